"""The operators that a serving loop runs next to the insert, the gather and
the pack, with their plain forms and the cases they are measured on:

* ``attention``  mla_latent_attention: new tokens of several sequences over
  their paged latent caches, in the absorbed form (every head of a token reads
  the same 576-wide rows; the first 512 columns are also the values);
* ``merge``      mla_merge_attn_states: attention results over disjoint parts
  of the context joined by their log-sum-exp;
* ``copy``       mla_cache_copy_blocks: pages copied, forked (a part of their
  rows) and cleared in every layer's cache.

``run`` computes the plain form with elementary torch operations in 32 bits
while ``own`` is false, and calls the library otherwise.
"""
import math
import random

import torch

own = False

RANK, ENTRY = 512, 576
SCALE = 192 ** -0.5  # the softmax scale of 128 + 64 wide heads before absorption
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
         "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


# ------------------------------------------------------------------ the cases
def _attention(name, seqs, q_len, kv_lo, kv_hi, heads, cache, block):
    c = {"op": "attention", "seqs": seqs, "q_len": q_len, "kv_lo": kv_lo, "kv_hi": kv_hi,
         "heads": heads, "cache": cache, "block": block}
    return dict(c, name=name) if name else c


def _merge(name, parts, tokens, heads, dim, dtype):
    c = {"op": "merge", "parts": parts, "tokens": tokens, "heads": heads, "dim": dim,
         "dtype": dtype}
    return dict(c, name=name) if name else c


def _copy(name, layers, copies, blocks, block, cache, partial):
    c = {"op": "copy", "layers": layers, "copies": copies, "blocks": blocks, "block": block,
         "cache": cache, "partial": partial}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user waiting for the next token: latency
        _attention("decode_1x2047_bf16", 1, 1, 2047, 2047, 16, "bf16", 64),
        # a full decode batch of mixed lengths over an fp8 cache
        _attention("decode_64_ragged_e4m3", 64, 1, 130, 16384, 16, "e4m3", 64),
        # long contexts: the cache's bytes are all that counts
        _attention("decode_4x131072_bf16", 4, 1, 131072, 131072, 16, "bf16", 64),
        # drafted tokens verified in one call, small pages
        _attention("verify_32x4_ragged_e5m2", 32, 4, 700, 8192, 16, "e5m2", 16),
        # all heads of a large model on one GPU: arithmetic and bytes are close
        _attention("decode_16_128heads_bf16", 16, 1, 1025, 8191, 128, "bf16", 64),
        # chunked prefill: new tokens over the context before them and each other
        _attention("chunk_2x1024_8k_bf16", 2, 1024, 8192, 8192, 16, "bf16", 64),
        # the suffix and the context of a decode batch joined
        _merge("merge_2x64_bf16", 2, 64, 16, 512, "bf16"),
        # the chunked-context loop's four partial results of an 8192-token chunk
        _merge("merge_4x8192_bf16", 4, 8192, 16, 128, "bf16"),
        # one sequence forked: its last, part-filled page in every layer
        _copy("fork_4_e4m3", 5, 4, 64, 64, "e4m3", True),
        # a cache compacted: a thousand whole pages moved in every layer
        _copy("compact_1024_bf16", 5, 1024, 2048, 64, "bf16", False),
        # many samples forked from their prompts, some freed pages cleared
        _copy("fork_512_e5m2", 5, 512, 2048, 64, "e5m2", True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "verify", "chunk", "merge", "copy"])
    cache = rng.choice(["bf16", "e4m3", "e5m2"])
    block = rng.choice([1, 16, 32, 48, 64, 64, 128])
    heads = rng.choice([1, 3, 8, 16, 16, 40, 64, 128])
    if op == "decode":
        seqs = _log(rng, 1, 256)
        hi = _log(rng, 1, min(131072, 400000 // seqs))
        return _attention(None, seqs, 1, _log(rng, 1, hi), hi, heads, cache, block)
    if op == "verify":
        seqs, q_len = _log(rng, 1, 64), rng.randint(2, 8)
        hi = _log(rng, q_len, min(32768, 200000 // seqs))
        return _attention(None, seqs, q_len, _log(rng, q_len, hi), hi, min(heads, 64), cache, block)
    if op == "chunk":
        seqs, q_len = rng.randint(1, 4), _log(rng, 17, 512)
        hi = q_len + _log(rng, 1, 7000)
        return _attention(None, seqs, q_len, q_len, hi, min(heads, 16), cache, block)
    if op == "merge":
        parts, heads, dim = rng.randint(2, 8), rng.choice([1, 3, 16, 24]), rng.choice([128, 192, 512])
        return _merge(None, parts, _log(rng, 1, min(16384, 60000000 // (parts * heads * dim))),
                      heads, dim, rng.choice(["bf16", "fp16", "fp32"]))
    blocks = _log(rng, 16, 2048)
    return _copy(None, rng.randint(1, 6), _log(rng, 1, blocks // 2), blocks,
                 rng.choice([16, 48, 64]), cache, rng.random() < 0.5)


def _kv_lens(c):
    """The sequences' lengths: spread evenly over [kv_lo, kv_hi], the longest among them."""
    lo, hi = c["kv_lo"], c["kv_hi"]
    return [hi] + [lo + int((hi - lo) * ((i * 0.6180339887) % 1.0)) for i in range(1, c["seqs"])]


def _copies(c):
    """(source, destination, rows) of each page copy: disjoint pages, some sources twice, some -1."""
    rng = random.Random(c["copies"] * 1000003 + c["blocks"])
    ids = rng.sample(range(c["blocks"]), 2 * c["copies"])
    src, dst = ids[:c["copies"]], ids[c["copies"]:]
    rows = [c["block"]] * c["copies"]
    if c["partial"]:
        for i in range(c["copies"]):
            rows[i] = rng.randint(0, c["block"])
            if i % 8 == 7:  # a freed page: cleared
                src[i], rows[i] = -1, c["block"]
            elif i % 4 == 1:
                src[i] = src[i - 1] if src[i - 1] >= 0 else src[i]
    return src, dst, rows


# ----------------------------------------------------------------- the inputs
def _cache(shape, kind, g, k_scale):
    """Latent rows ~ N(0, 1), stored as the insert stores them (fp8: divided by k_scale)."""
    out = torch.empty(shape, dtype=TYPES[kind], device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):  # in parts: the largest cache is several GB in fp32
        n = min(1 << 28, flat.numel() - i)
        x = torch.randn(n, generator=g, device="cuda")
        flat[i:i + n] = (x if kind == "bf16" else (x / k_scale).clamp_(-448, 448)).to(TYPES[kind])
    return out


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "attention":
        lens = _kv_lens(c)
        pages = [(n + c["block"] - 1) // c["block"] for n in lens]
        blocks, width = sum(pages) + 3, max(pages)
        perm = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(c["seqs"], width, dtype=torch.int32)
        used, host = 0, perm.cpu()
        for i, p in enumerate(pages):
            table[i, :p] = host[used:used + p]
            used += p
        k_scale = 0.01 + 0.005 * float(torch.rand(1, generator=g, device="cuda"))
        tokens = c["seqs"] * c["q_len"]
        s.update(
            cache=_cache((blocks, c["block"], ENTRY), c["cache"], g, k_scale),
            k_scale=None if c["cache"] == "bf16" else torch.tensor([k_scale], device="cuda"),
            table=table.cuda(), kv_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
            cu=torch.arange(0, tokens + 1, c["q_len"], dtype=torch.int32, device="cuda"),
            q=torch.randn(tokens, c["heads"], ENTRY, generator=g, device="cuda").bfloat16(),
            out=torch.empty(tokens, c["heads"], RANK, dtype=torch.bfloat16, device="cuda"),
            lse=torch.empty(tokens, c["heads"], dtype=torch.float32, device="cuda"))
    elif c["op"] == "merge":
        shape = (c["parts"], c["tokens"], c["heads"])
        lse = 8.0 + 1.5 * torch.randn(shape, generator=g, device="cuda")
        # one in sixteen rows has a part whose mask left nothing
        lse[torch.rand(shape, generator=g, device="cuda") < 1 / 16] = -math.inf
        x = torch.randn(*shape, c["dim"], generator=g, device="cuda")
        x[lse == -math.inf] = 0.0
        s.update(parts=x.to(TYPES[c["dtype"]]), lse=lse,
                 out=torch.empty(shape[1:] + (c["dim"],), dtype=TYPES[c["dtype"]], device="cuda"),
                 lse_out=torch.empty(shape[1:], device="cuda"))
    else:
        src, dst, rows = _copies(c)
        dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        cache = _cache((c["layers"], c["blocks"], c["block"], ENTRY), c["cache"], g, 0.01)
        cache = cache.view(torch.int16 if c["cache"] == "bf16" else torch.uint8)
        s.update(cache=cache, src=dev(src), dst=dev(dst), rows=dev(rows),
                 ptrs=torch.tensor([cache[i].data_ptr() for i in range(c["layers"])],
                                   dtype=torch.int64, device="cuda"))
    if own:
        from pack_mla_cache_gb300 import ops
        s["ops"] = ops
        if c["op"] == "attention":  # a program keeps one workspace for all its calls
            n = ops.mla_latent_attention_workspace(c["seqs"] * c["q_len"], c["heads"], c["seqs"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------- one pass
def _own_attention(s, c):
    s["ops"].mla_latent_attention(
        s["q"][:, :, :RANK], s["q"][:, :, RANK:], s["cache"], s["cache"].dtype,
        s["cache"].shape[0], c["block"], c["block"] * ENTRY, ENTRY, s["table"], s["cu"],
        s["kv_lens"], s["out"], s["ws"], lse=s["lse"], softmax_scale=SCALE, k_scale=s["k_scale"],
        causal=True)
    return s["out"], s["lse"]


def _plain_attention(s, c):
    n, heads, width = c["seqs"], c["heads"], c["kv_hi"]
    pos = torch.arange(width, device="cuda")
    block = s["table"].long()[:, pos // c["block"]]              # [n, width]
    raw = s["cache"].view(torch.int16 if c["cache"] == "bf16" else torch.uint8)
    kv = raw[block, (pos % c["block"])[None]].view(s["cache"].dtype).float()  # [n, width, 576]
    if s["k_scale"] is not None:
        kv = kv * s["k_scale"]
    q = s["q"].float().view(n, c["q_len"] * heads, ENTRY)
    x = torch.matmul(q, kv.transpose(1, 2)).mul_(SCALE)          # [n, q_len * heads, width]
    first_hidden = s["kv_lens"].long()[:, None] - c["q_len"] + 1 \
        + torch.arange(c["q_len"], device="cuda")[None]          # [n, q_len]
    hidden = pos[None, None] >= first_hidden[:, :, None]
    x.view(n, c["q_len"], heads, width).masked_fill_(hidden[:, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x.sub_(top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, kv[:, :, :RANK]) / total
    s["out"].copy_(out.view(s["out"].shape))
    s["lse"].copy_((top + torch.log(total)).view(s["lse"].shape))
    return s["out"], s["lse"]


def _own_merge(s, c):
    s["ops"].mla_merge_attn_states(s["parts"], s["lse"], s["out"], lse_out=s["lse_out"])
    return s["out"], s["lse_out"]


def _plain_merge(s, c):
    top = s["lse"].amax(0)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    w = torch.exp(s["lse"] - top)
    total = w.sum(0)
    mean = (w[..., None] * s["parts"].float()).sum(0) / torch.where(total > 0, total, 1.0)[..., None]
    s["out"].copy_(mean)
    s["lse_out"].copy_(top + torch.log(total))
    return s["out"], s["lse_out"]


def _own_copy(s, c):
    s["ops"].mla_cache_copy_blocks(s["ptrs"], TYPES[c["cache"]], c["blocks"], c["block"],
                                   c["block"] * ENTRY, ENTRY, ENTRY, s["src"], s["dst"],
                                   row_counts=s["rows"])
    return s["cache"]


def _plain_copy(s, c):
    src, dst = s["src"].long(), s["dst"].long()
    new = s["cache"][:, src.clamp(min=0)]
    new.masked_fill_((src < 0)[None, :, None, None], 0)
    kept = torch.arange(c["block"], device="cuda")[None] >= s["rows"][:, None]
    s["cache"][:, dst] = torch.where(kept[None, :, :, None], s["cache"][:, dst], new)
    return s["cache"]


def run(state):
    c = state["case"]
    if own:
        return {"attention": _own_attention, "merge": _own_merge, "copy": _own_copy}[c["op"]](state, c)
    return {"attention": _plain_attention, "merge": _plain_merge, "copy": _plain_copy}[c["op"]](state, c)


# ------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    size = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1, "e5m2": 1}
    if c["op"] == "attention":
        lens, rows = _kv_lens(c), c["seqs"] * c["q_len"] * c["heads"]
        # token j of a sequence sees kv_len - q_len + 1 + j rows
        pairs = sum(c["q_len"] * (n - c["q_len"] + 1) + c["q_len"] * (c["q_len"] - 1) // 2
                    for n in lens) * c["heads"]
        table = sum((n + c["block"] - 1) // c["block"] for n in lens) * 4 + 8 * c["seqs"]
        return {"bytes": sum(lens) * ENTRY * size[c["cache"]] + rows * (ENTRY * 2 + RANK * 2 + 4)
                + table, "flops": 2 * pairs * (ENTRY + RANK)}
    if c["op"] == "merge":
        rows = c["tokens"] * c["heads"]
        return {"bytes": rows * ((c["parts"] + 1) * (c["dim"] * size[c["dtype"]] + 4)),
                "flops": 2 * rows * c["parts"] * c["dim"]}
    src, dst, rows = _copies(c)
    moved = sum(r * (2 if s >= 0 else 1) for s, r in zip(src, rows))
    return {"bytes": moved * c["layers"] * ENTRY * size[c["cache"]] + 12 * c["copies"], "flops": 0}


# --------------------------------------------------------------------- 64 bits
def exact(case, seed):
    c = case
    if c["op"] == "copy":
        return None
    s = prepare(c, seed)
    if c["op"] == "merge":
        lse, parts = s["lse"].double(), s["parts"].double()
        whole = torch.logsumexp(lse, 0)
        share = torch.exp(lse - torch.where(whole == -math.inf, 0.0, whole))
        return torch.einsum("pth,pthd->thd", share, parts), whole
    outs, lses = [], []
    for i, n in enumerate(_kv_lens(c)):  # one sequence at a time, its rows from its own pages
        pages = s["table"][i, :(n + c["block"] - 1) // c["block"]].long()
        raw = s["cache"].view(torch.int16 if c["cache"] == "bf16" else torch.uint8)
        kv = raw[pages].view(s["cache"].dtype).reshape(-1, ENTRY)[:n].double()
        if s["k_scale"] is not None:
            kv = kv * s["k_scale"].double()
        for t in range(0, c["q_len"], 128):
            t1 = min(t + 128, c["q_len"])
            q = s["q"][i * c["q_len"] + t:i * c["q_len"] + t1].double()
            logits = torch.einsum("the,ke->thk", q, kv) * SCALE
            seen = torch.arange(n, device="cuda")[None] <= \
                torch.arange(n - c["q_len"] + t, n - c["q_len"] + t1, device="cuda")[:, None]
            logits = torch.where(seen[:, None], logits, -math.inf)
            outs.append(torch.einsum("thk,ke->the", torch.softmax(logits, -1), kv[:, :RANK]))
            lses.append(torch.logsumexp(logits, -1))
    return torch.cat(outs), torch.cat(lses)
