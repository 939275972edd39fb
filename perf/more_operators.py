"""The operators around prompts and drafted trees, with their plain forms and the cases they
are measured on:

* ``prefill``  mla_prefill_attention: packed sequences (whole prompts, chunks of new tokens,
  single tokens) over keys and values per head, as the chunked-context pack writes them or
  as kv_b_proj leaves them;
* ``tree``     mla_latent_tree_attention: trees of drafted tokens verified over the paged
  latent caches, each token seeing the context and its ancestors;
* ``compact``  mla_cache_compact_rows: the rows of the accepted branch moved to the front of
  the drafted ones in every layer's cache.

``run`` computes the plain form with elementary torch operations in 32 bits while ``own`` is
false, and calls the library otherwise.
"""
import math
import random

import torch

own = False

RANK, ENTRY = 512, 576      # latent rows: 512 + 64
NOPE, ROPE, V = 128, 64, 128  # heads after kv_b_proj
SCALE = (NOPE + ROPE) ** -0.5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16,
         "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
SIZE = {"bf16": 2, "fp16": 2, "e4m3": 1, "e5m2": 1}


# ------------------------------------------------------------------ the cases
def _prefill(name, seqs, q_lo, q_hi, ctx_lo, ctx_hi, causal, heads, kv_heads, dtype, kv, packed):
    """New tokens q_lo..q_hi a sequence; causal: behind ctx rows of context, else over them alone."""
    c = {"op": "prefill", "seqs": seqs, "q_lo": q_lo, "q_hi": q_hi, "ctx_lo": ctx_lo,
         "ctx_hi": ctx_hi, "causal": causal, "heads": heads, "kv_heads": kv_heads,
         "dtype": dtype, "kv": kv, "packed": packed}
    return dict(c, name=name) if name else c


def _tree(name, seqs, n_lo, n_hi, kv_lo, kv_hi, heads, cache, block):
    c = {"op": "tree", "seqs": seqs, "n_lo": n_lo, "n_hi": n_hi, "kv_lo": kv_lo, "kv_hi": kv_hi,
         "heads": heads, "cache": cache, "block": block}
    return dict(c, name=name) if name else c


def _compact(name, layers, seqs, drafted, accepted, cache, block):
    c = {"op": "compact", "layers": layers, "seqs": seqs, "drafted": drafted,
         "accepted": accepted, "cache": cache, "block": block}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a short prompt on its own: latency
        _prefill("prompt_1x300_bf16", 1, 300, 300, 0, 0, True, 16, 16, "bf16", "bf16", True),
        # a prefill batch of mixed prompts, keys and values read where kv_b_proj left them
        _prefill("prompts_16_ragged_bf16", 16, 37, 2048, 0, 0, True, 16, 16, "bf16", "bf16", False),
        # one long prompt: arithmetic is all that counts
        _prefill("prompt_1x16384_bf16", 1, 16384, 16384, 0, 0, True, 16, 16, "bf16", "bf16", True),
        # one step of the chunked-context loop: new tokens over a packed fp8 chunk of context
        _prefill("context_2x1024_8k_e4m3", 2, 1024, 1024, 8192, 8192, False, 16, 16, "bf16", "e4m3", True),
        # prompts behind cached prefixes, several query heads to a key head
        _prefill("grouped_4_ragged_fp16", 4, 700, 1501, 130, 2100, True, 32, 4, "fp16", "fp16", True),
        # single tokens over expanded context: bytes are all that counts
        _prefill("tokens_32_ragged_bf16", 32, 1, 1, 500, 4096, True, 16, 16, "bf16", "bf16", True),
        # one user's small tree: latency
        _tree("tree_1x8_bf16", 1, 8, 8, 2047, 2047, 16, "bf16", 64),
        # a batch of trees of different sizes over an fp8 cache with small pages
        _tree("trees_32x16_ragged_e4m3", 32, 5, 16, 700, 8192, 16, "e4m3", 16),
        # wide trees over bf16 caches
        _tree("trees_16x61_bf16", 16, 61, 61, 1025, 8191, 16, "bf16", 64),
        # one user's accepted branch
        _compact("accept_1x5_e4m3", 5, 1, 16, 5, "e4m3", 64),
        # a large batch's
        _compact("accept_512x9_bf16", 5, 512, 61, 9, "bf16", 64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "context", "tokens", "tree", "tree", "compact"])
    block = rng.choice([1, 16, 32, 48, 64, 64, 128])
    cache = rng.choice(["bf16", "e4m3", "e5m2"])
    if op in ("prompt", "context", "tokens"):
        kv_heads = rng.choice([1, 2, 4, 8, 16])
        heads = kv_heads * rng.choice([1, 1, 1, 2, 3, 8]) if kv_heads < 8 else kv_heads
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        kv = rng.choice([dtype, dtype, "e4m3", "e5m2"])
        packed = rng.random() < 0.5
        # padded pairs of the plain form: at most a quarter of the longest prompt's
        room = 2 ** 30 // heads
        if op == "tokens":
            seqs, q_hi = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4])
            hi = _log(rng, 1, min(16384, 65536 // seqs))
            return _prefill(None, seqs, 1, q_hi, _log(rng, 1, hi), hi, rng.random() < 0.5, heads,
                            kv_heads, dtype, kv, packed)
        seqs = _log(rng, 1, 32)
        most = int((room // seqs) ** 0.5)
        q_hi = _log(rng, 1, min(8192, most))
        q_lo = _log(rng, 1, q_hi)
        causal = op == "prompt"
        hi = max(0 if causal else 1, min(8192, room // seqs // q_hi - (q_hi if causal else 0)))
        hi = rng.choice([0, _log(rng, 1, hi)]) if causal and hi > 0 else hi and _log(rng, 1, hi)
        return _prefill(None, seqs, q_lo, q_hi, hi and _log(rng, 1, hi), hi, causal, heads,
                        kv_heads, dtype, kv, packed)
    if op == "tree":
        seqs, n_hi = _log(rng, 1, 64), _log(rng, 2, 64)
        hi = n_hi + _log(rng, 1, min(32768, 200000 // seqs))
        return _tree(None, seqs, rng.randint(1, n_hi), n_hi, n_hi + _log(rng, 1, hi - n_hi), hi,
                     rng.choice([1, 3, 8, 16, 16, 40] + [128] * (seqs < 17)), cache, block)
    drafted = _log(rng, 2, 64)
    return _compact(None, rng.randint(1, 6), _log(rng, 1, 512), drafted,
                    rng.randint(1, min(16, drafted)), cache, block)


def _spread(lo, hi, n):
    """n lengths spread evenly over [lo, hi], the longest first."""
    return [hi] + [lo + int((hi - lo) * ((i * 0.6180339887) % 1.0)) for i in range(1, n)]


def _lens(c):
    """(new tokens, rows seen by the last of them) of each sequence of a prefill or tree case."""
    if c["op"] == "tree":
        return _spread(c["n_lo"], c["n_hi"], c["seqs"]), _spread(c["kv_lo"], c["kv_hi"], c["seqs"])
    q = _spread(c["q_lo"], c["q_hi"], c["seqs"])
    ctx = _spread(c["ctx_lo"], c["ctx_hi"], c["seqs"])[::-1]  # long prompts behind short contexts
    return q, [x + n if c["causal"] else x for x, n in zip(ctx, q)]


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


# ----------------------------------------------------------------- the inputs
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _stored(shape, kind, g, scale):
    """Values ~ N(0, 1) as a cache or a pack stores them (fp8: divided by the scale)."""
    x = torch.randn(shape, generator=g, device="cuda")
    return x.to(TYPES[kind]) if SIZE[kind] == 2 else (x / scale).clamp_(-448, 448).to(TYPES[kind])


def _pages(lens, block, spare, g):
    """A block table over shuffled blocks, and how many blocks there are."""
    pages = [(n + block - 1) // block for n in lens]
    blocks = sum(pages) + spare
    host = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.zeros(len(lens), max(pages), dtype=torch.int32)
    used = 0
    for i, p in enumerate(pages):
        table[i, :p] = host[used:used + p]
        used += p
    return table.cuda(), blocks


def _trees(c, seed):
    """Ancestor masks (own bit included) of random trees as int32 words [tokens, words]."""
    rng = random.Random(seed * 7919 + 5)
    words = (c["n_hi"] + 31) // 32
    rows = []
    for n in _lens(c)[0]:
        seen = []
        for i in range(n):
            up = rng.randint(-1, i - 1) if rng.random() < 0.5 else i - 1  # long and short branches
            seen.append((seen[up] if up >= 0 else 0) | 1 << i)
        for m in seen:
            w = [m >> 32 * k & 0xFFFFFFFF for k in range(words)]
            rows.append([x - (1 << 32) if x >> 31 else x for x in w])
    return _ints(rows)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    scale = 0.01 + 0.005 * float(torch.rand(1, generator=g, device="cuda"))
    if c["op"] == "prefill":
        q_lens, kv_lens = _lens(c)
        T, K, H, G = sum(q_lens), sum(kv_lens), c["heads"], c["kv_heads"]
        dt, kv = TYPES[c["dtype"]], c["kv"]
        q = (1.5 * torch.randn(T, H, NOPE + ROPE, generator=g, device="cuda")).to(dt)
        if c["packed"]:  # the pack's output: whole keys, contiguous values
            key = _stored((K, G, NOPE + ROPE), kv, g, scale)
            key.view(torch.uint8 if SIZE[kv] == 1 else torch.int16)[:, :, NOPE:] = \
                key.view(torch.uint8 if SIZE[kv] == 1 else torch.int16)[:, :1, NOPE:].clone()
            k_nope, k_pe, v = key[:, :, :NOPE], key[:, :, NOPE:], _stored((K, G, V), kv, g, scale)
        else:  # kv_b_proj's output and one rotary row for all heads
            both = _stored((K, G, NOPE + V), kv, g, scale)
            k_nope, v, k_pe = both[:, :, :NOPE], both[:, :, NOPE:], _stored((K, ROPE), kv, g, scale)
        s.update(q=q, k_nope=k_nope, k_pe=k_pe, v=v, cu_q=_ints(_cu(q_lens)), cu_kv=_ints(_cu(kv_lens)),
                 kv_scale=torch.tensor([scale], device="cuda") if SIZE[kv] == 1 else None,
                 out=torch.empty(T, H, V, dtype=dt, device="cuda"),
                 lse=torch.empty(T, H, dtype=torch.float32, device="cuda"))
    elif c["op"] == "tree":
        n, kv_lens = _lens(c)
        table, blocks = _pages(kv_lens, c["block"], 3, g)
        T = sum(n)
        s.update(cache=_stored((blocks, c["block"], ENTRY), c["cache"], g, scale), table=table,
                 k_scale=None if c["cache"] == "bf16" else torch.tensor([scale], device="cuda"),
                 kv_lens=_ints(kv_lens), cu_q=_ints(_cu(n)), mask=_trees(c, seed),
                 q=torch.randn(T, c["heads"], ENTRY, generator=g, device="cuda").bfloat16(),
                 out=torch.empty(T, c["heads"], RANK, dtype=torch.bfloat16, device="cuda"),
                 lse=torch.empty(T, c["heads"], dtype=torch.float32, device="cuda"))
    else:
        rng = random.Random(seed * 104729 + 11)
        starts = [rng.randint(0, 3 * c["block"]) for _ in range(c["seqs"])]
        rows, counts = [], []
        for _ in starts:  # an increasing branch of the drafted rows
            k = rng.randint(1, c["accepted"])
            rows.append(sorted(rng.sample(range(c["drafted"]), k)) + [0] * (c["accepted"] - k))
            counts.append(k)
        counts[0] = c["accepted"]
        rows[0] = sorted(rng.sample(range(c["drafted"]), c["accepted"]))
        table, blocks = _pages([3 * c["block"] + c["drafted"]] * c["seqs"], c["block"], 2, g)
        cache = _stored((c["layers"], blocks, c["block"], ENTRY), c["cache"], g, scale)
        cache = cache.view(torch.int16 if c["cache"] == "bf16" else torch.uint8)
        s.update(cache=cache, table=table, starts=_ints(starts), rows=_ints(rows), counts=_ints(counts),
                 ptrs=torch.tensor([cache[i].data_ptr() for i in range(c["layers"])],
                                   dtype=torch.int64, device="cuda"))
    if own:
        from pack_mla_cache_gb300 import ops
        s["ops"] = ops
        if c["op"] == "prefill":  # a program keeps one workspace for all its calls
            n = ops.mla_prefill_attention_workspace(T, c["heads"], c["kv_heads"], c["seqs"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        if c["op"] == "tree":
            n = ops.mla_latent_attention_workspace(T, c["heads"], c["seqs"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------- one pass
def _own_prefill(s, c):
    s["ops"].mla_prefill_attention(
        s["q"][:, :, :NOPE], s["q"][:, :, NOPE:], s["k_nope"], s["k_pe"], s["v"], s["cu_q"],
        s["cu_kv"], s["out"], s["ws"], softmax_scale=SCALE, causal=c["causal"],
        kv_scale=s["kv_scale"], lse=s["lse"])
    return s["out"], s["lse"]


def _softmax(x, v):
    """(weights of x) * v and the log-sum-exp, a row that sees nothing 0 and -inf; x is used up."""
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    return out, (top + torch.log(total))[..., 0]


def _padded(cu, width, limit):
    """[seqs, width] row numbers of packed sequences, and whether each row exists."""
    at = cu[:-1].long()[:, None] + torch.arange(width, device="cuda")[None]
    return at.clamp(max=limit - 1), at < cu[1:].long()[:, None]


def _plain_prefill(s, c):
    q_lens, kv_lens = _lens(c)
    n, L, M, H, G = c["seqs"], max(q_lens), max(kv_lens), c["heads"], c["kv_heads"]
    T, K = s["q"].shape[0], s["k_nope"].shape[0]
    qi, q_in = _padded(s["cu_q"], L, T)
    ki, k_in = _padded(s["cu_kv"], M, K)
    k_pe = s["k_pe"].float()
    k_pe = k_pe if k_pe.dim() == 3 else k_pe[:, None].expand(K, G, ROPE)
    key = torch.cat([s["k_nope"].float(), k_pe], -1)[ki].permute(0, 2, 3, 1)  # [n, G, 192, M]
    v = s["v"].float()[ki].permute(0, 2, 1, 3)                               # [n, G, M, 128]
    if s["kv_scale"] is not None:
        key, v = key * s["kv_scale"], v * s["kv_scale"]
    q = s["q"].float()[qi].view(n, L, G, H // G, NOPE + ROPE).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(n, G, H // G * L, NOPE + ROPE), key).mul_(SCALE)
    hidden = ~k_in[:, None]                                                   # [n, L, M]
    if c["causal"]:
        nq = (s["cu_q"][1:] - s["cu_q"][:-1]).long()[:, None, None]
        nk = (s["cu_kv"][1:] - s["cu_kv"][:-1]).long()[:, None, None]
        pos = torch.arange(M, device="cuda")[None, None]
        hidden = hidden | (pos > nk - nq + torch.arange(L, device="cuda")[None, :, None])
    else:
        hidden = hidden.expand(n, L, M)
    x.view(n, G, H // G, L, M).masked_fill_(hidden[:, None, None], -math.inf)
    out, lse = _softmax(x, v)
    out = out.view(n, H, L, V).transpose(1, 2)[q_in]    # packed again: [T, H, 128]
    s["out"].copy_(out)
    s["lse"].copy_(lse.view(n, H, L).transpose(1, 2)[q_in])
    return s["out"], s["lse"]


def _own_tree(s, c):
    s["ops"].mla_latent_tree_attention(
        s["q"][:, :, :RANK], s["q"][:, :, RANK:], s["cache"], s["cache"].dtype,
        s["cache"].shape[0], c["block"], c["block"] * ENTRY, ENTRY, s["table"], s["cu_q"],
        s["kv_lens"], s["mask"], s["out"], s["ws"], lse=s["lse"], softmax_scale=SCALE,
        k_scale=s["k_scale"])
    return s["out"], s["lse"]


def _plain_tree(s, c):
    n, H, width, L = c["seqs"], c["heads"], c["kv_hi"], c["n_hi"]
    pos = torch.arange(width, device="cuda")
    block = s["table"].long()[:, pos // c["block"]]              # [n, width]
    raw = s["cache"].view(torch.int16 if c["cache"] == "bf16" else torch.uint8)
    kv = raw[block, (pos % c["block"])[None]].view(s["cache"].dtype).float()  # [n, width, 576]
    if s["k_scale"] is not None:
        kv = kv * s["k_scale"]
    qi, q_in = _padded(s["cu_q"], L, s["q"].shape[0])
    q = s["q"].float()[qi]                                       # [n, L, H, 576]
    x = torch.matmul(q.view(n, L * H, ENTRY), kv.transpose(1, 2)).mul_(SCALE)
    first_new = s["kv_lens"].long() - (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    node = pos[None] - first_new[:, None]                        # [n, width]: number of a new row
    word = (node.clamp(min=0) >> 5).clamp(max=s["mask"].shape[1] - 1)
    mine = s["mask"][qi]                                         # [n, L, words]
    bits = torch.gather(mine, 2, word[:, None].expand(n, L, width)).long() >> (node[:, None] & 31)
    seen = (node[:, None] < 0) | ((bits & 1) != 0)
    seen &= (pos[None] < s["kv_lens"].long()[:, None])[:, None]
    x.view(n, L, H, width).masked_fill_(~seen[:, :, None], -math.inf)
    out, lse = _softmax(x, kv[:, :, :RANK])
    s["out"].copy_(out.view(n, L, H, RANK)[q_in])
    s["lse"].copy_(lse.view(n, L, H)[q_in])
    return s["out"], s["lse"]


def _own_compact(s, c):
    s["ops"].mla_cache_compact_rows(s["ptrs"], TYPES[c["cache"]], s["cache"].shape[1], c["block"],
                                    c["block"] * ENTRY, ENTRY, ENTRY, s["table"], s["starts"],
                                    s["rows"], s["counts"])
    return s["cache"]


def _plain_compact(s, c):
    i = torch.arange(c["accepted"], device="cuda")[None]
    live = i < s["counts"][:, None]
    seq = torch.arange(c["seqs"], device="cuda")[:, None].expand_as(live)[live]
    to = (s["starts"][:, None] + i)[live].long()
    src = (s["starts"][:, None] + s["rows"])[live].long()
    table = s["table"].long()
    moved = s["cache"][:, table[seq, src // c["block"]], src % c["block"]]
    s["cache"][:, table[seq, to // c["block"]], to % c["block"]] = moved
    return s["cache"]


def run(state):
    c = state["case"]
    if own:
        return {"prefill": _own_prefill, "tree": _own_tree, "compact": _own_compact}[c["op"]](state, c)
    return {"prefill": _plain_prefill, "tree": _plain_tree, "compact": _plain_compact}[c["op"]](state, c)


# ------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "compact":  # about half of the longest branches; every row read and written once
        rows = c["seqs"] * (c["accepted"] + 1) / 2
        return {"bytes": 2 * rows * c["layers"] * ENTRY * SIZE[c["cache"]]
                + c["seqs"] * (8 + 4 * c["accepted"]), "flops": 0}
    q_lens, kv_lens = _lens(c)
    T, H = sum(q_lens), c["heads"]
    if c["op"] == "tree":  # every drafted token sees the context and at most its tree
        pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(q_lens, kv_lens)) * H
        table = sum((m + c["block"] - 1) // c["block"] for m in kv_lens) * 4 + 8 * c["seqs"]
        return {"bytes": sum(kv_lens) * ENTRY * SIZE[c["cache"]] + T * H * (ENTRY * 2 + RANK * 2 + 4)
                + T * ((c["n_hi"] + 31) // 32) * 4 + table, "flops": 2 * pairs * (ENTRY + RANK)}
    pairs = H * sum(n * m - (n * (n - 1) // 2 if c["causal"] else 0) for n, m in zip(q_lens, kv_lens))
    per_row = c["kv_heads"] * (NOPE + V) + (c["kv_heads"] if c["packed"] else 1) * ROPE
    return {"bytes": T * H * (2 * (NOPE + ROPE + V) + 4) + sum(kv_lens) * per_row * SIZE[c["kv"]]
            + 8 * (c["seqs"] + 1), "flops": 2 * pairs * (NOPE + ROPE + V)}


# --------------------------------------------------------------------- 64 bits
def _attend64(q, key, v, seen):
    """q [t, H, e], key / v [k, H or 1, .], seen [t, k]: out [t, H, .] and lse [t, H]."""
    logits = torch.einsum("the,khe->thk", q, key.expand(-1, q.shape[1], -1)) * SCALE
    logits = torch.where(seen[:, None], logits, -math.inf)
    lse = torch.logsumexp(logits, -1)
    w = torch.exp(logits - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    return torch.einsum("thk,khe->the", w, v.expand(-1, q.shape[1], -1)), lse


def exact(case, seed):
    c = case
    if c["op"] == "compact":
        return None
    s = prepare(c, seed)
    q_lens, kv_lens = _lens(c)
    cq, ck = _cu(q_lens), _cu(kv_lens)
    outs, lses = [], []
    for i, (n, m) in enumerate(zip(q_lens, kv_lens)):  # one sequence at a time
        if c["op"] == "tree":  # its rows from its own pages
            pages = s["table"][i, :(m + c["block"] - 1) // c["block"]].long()
            raw = s["cache"].view(torch.int16 if c["cache"] == "bf16" else torch.uint8)
            key = raw[pages].view(s["cache"].dtype).reshape(-1, 1, ENTRY)[:m].double()
            key = key if s["k_scale"] is None else key * s["k_scale"].double()
            v = key[:, :, :RANK]
        else:
            rows = slice(ck[i], ck[i + 1])
            pe = s["k_pe"][rows].double()
            pe = pe if pe.dim() == 3 else pe[:, None].expand(m, c["kv_heads"], ROPE)
            key, v = torch.cat([s["k_nope"][rows].double(), pe], -1), s["v"][rows].double()
            if s["kv_scale"] is not None:
                key, v = key * s["kv_scale"].double(), v * s["kv_scale"].double()
            share = c["heads"] // c["kv_heads"]
            key, v = key.repeat_interleave(share, 1), v.repeat_interleave(share, 1)
        for t in range(0, n, 256):
            t1 = min(t + 256, n)
            pos = torch.arange(m, device="cuda")[None]
            if c["op"] == "tree":
                node = pos - (m - n)
                word = s["mask"][cq[i] + t:cq[i] + t1].long() & 0xFFFFFFFF
                bit = word[:, node[0].clamp(min=0) // 32] >> (node.clamp(min=0) % 32) & 1
                seen, last = (node < 0) | (bit == 1), m
            elif c["causal"]:
                seen = pos <= m - n + torch.arange(t, t1, device="cuda")[:, None]
                last = max(1, m - n + t1) if m else 0
            else:
                seen, last = (pos >= 0).expand(t1 - t, m), m
            o, le = _attend64(s["q"][cq[i] + t:cq[i] + t1].double(), key[:last], v[:last],
                              seen[:, :last])
            outs.append(o)
            lses.append(le)
    return torch.cat(outs), torch.cat(lses)
