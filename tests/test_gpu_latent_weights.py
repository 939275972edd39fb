"""The softmax weights of mla_latent_attention: 8 bits of every weight, whatever
its size, and results that do not depend on how a call is cut over the SMs.

Each case is one early row that takes much of the weight (5 to 14 nats above the
others, one gap per head) and a long tail of equal scores whose values are all
positive, so that errors of the weights add up instead of averaging out.  A batch of
as many equal sequences as the GPU has SMs puts each of them, sink and tail, into
one CTA's run; a sequence alone is cut into many."""
import numpy as np
import pytest
import torch

import devutil as D
import refattn as R
from pack_mla_cache_gb300 import ops

pytestmark = pytest.mark.gpu
PAGE, K_SCALE = 64, 2.0 ** -6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pack_mla_cache_gb300 import build
    build.build()
    ops.lib()


class Sink:
    """Page 0: the sink (values around `sink`) and 63 tail rows; page 1: 64 tail rows, as often as asked."""

    def __init__(self, fmt, heads, rows, sink, seed=5):
        rng = np.random.default_rng(seed)
        x = rng.uniform(0.5, 1.5, (2 * PAGE, R.ENTRY))
        x[0, :R.RANK] += sink - 1
        x[:, R.RANK:] = 0
        x[0, R.RANK] = 1   # the gap's column
        x[:, R.RANK + 1] = 1
        x = x.astype(np.float32)
        self.fmt, self.heads, self.rows = fmt, heads, rows
        if fmt == 0:
            codes = R.orc.bf16_from_f32_array(x)
            self.values = R.orc.bf16_bits_to_f64(codes).reshape(x.shape)
            self.cache, self.k_scale = D.dev_bf16(codes), None
        else:
            codes = R.orc.fp8_encode(x / np.float32(K_SCALE), fmt).reshape(x.shape)
            lut = R.orc.fp8_decode(np.arange(256, dtype=np.uint8), fmt)
            self.values = np.asarray(lut)[codes] * K_SCALE
            self.cache = D.dev(codes)
            self.k_scale = torch.tensor([K_SCALE], device="cuda")
        q = np.zeros((heads, R.ENTRY), np.float32)
        q[:, R.RANK] = np.linspace(5, 14, heads) / R.SCALE
        q[:, R.RANK + 1] = np.linspace(-3.3, 4.1, heads) / R.SCALE
        self.q = R.orc.bf16_from_f32_array(q)

    def run(self, seqs):
        """(out, lse) of `seqs` sequences of one token over the same pages."""
        dev, heads = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda"), self.heads
        table = dev([0] + [1] * (self.rows // PAGE - 1)).expand(seqs, -1).contiguous()
        q = D.dev_bf16(self.q).view(1, heads, R.ENTRY).expand(seqs, -1, -1)
        out = torch.empty(seqs, heads, R.RANK, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(seqs, heads, device="cuda")
        ws = torch.empty(ops.mla_latent_attention_workspace(seqs, heads, seqs), dtype=torch.uint8,
                         device="cuda")
        ops.mla_latent_attention(q[:, :, :512], q[:, :, 512:], self.cache, self.fmt, 2, PAGE,
                                 PAGE * R.ENTRY, R.ENTRY, table, dev(list(range(seqs + 1))),
                                 dev([self.rows] * seqs), out, ws, softmax_scale=R.SCALE,
                                 k_scale=self.k_scale, lse=lse)
        torch.cuda.synchronize()
        return out, lse

    def exact(self):
        """out [heads, 512], lse [heads] in float64 and how far a result may be from them.

        The bound counts what the interface states: 2^-8 of every weight, scores off by
        at most d = 576 fp32 steps of the sum of magnitudes (and, with an fp8 cache, 2^-21
        of the query row's largest element per element), sums off by two steps of 2^-23
        per row, fp32 exponentials (2^-18 in all), one rounding of the result."""
        qv, v = R.orc.bf16_bits_to_f64(self.q).reshape(self.heads, R.ENTRY), self.values
        x = R.SCALE * (qv @ v.T)                                    # [heads, 128]
        times = np.ones(2 * PAGE)
        times[PAGE:] = self.rows // PAGE - 1
        top = x.max(-1, keepdims=True)
        w = np.exp(x - top) * times
        total = w.sum(-1, keepdims=True)
        out, mag = (w / total) @ v[:, :R.RANK], (w / total) @ np.abs(v[:, :R.RANK])
        d = 576 * 2.0 ** -23 * R.SCALE * (np.abs(qv) @ np.abs(v).T).max(-1)
        if self.fmt:
            d = d + 2.0 ** -21 * R.SCALE * np.abs(qv).max(-1) * np.abs(v).sum(-1).max()
        sums = 2 * self.rows * 2.0 ** -23 + 2.0 ** -18
        err = (R.BF16_HALF + 4 * d + sums)[:, None] * mag
        lse = (top + np.log(total))[:, 0]
        return out, lse, err + R.BF16_HALF * (np.abs(out) + err), d + sums + 2.0 ** -22 * np.abs(lse)


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("rows", [2048, 16384, 131072])
@pytest.mark.parametrize("heads", [16, 32, 64])
@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_a_long_tail_behind_a_sink(fmt, heads, rows):
    s = Sink(fmt, heads, rows, -1)
    ro, rl, bo, bl = s.exact()
    for seqs in (sms(), 1):
        out, lse = s.run(seqs)
        assert (out == out[0]).all() and (lse == lse[0]).all()
        o, le = out[0].double().cpu().numpy(), lse[0].double().cpu().numpy()
        worst = (np.abs(o - ro) / bo).max(-1)
        assert worst.max() <= 1, (seqs, worst)
        assert (np.abs(le - rl) <= bl).all()


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_the_cut_over_the_sms_does_not_change_the_weights(fmt, heads):
    """In one run and cut into sixteen, the weights round alike: what differs are fp32
    sums.  2048 rows are 32 tiles, 128 additions of a matrix unit at most, each off by one
    fp32 step: a relative 2^-16, against steps of the bf16 result of 2^-8 and more.  A
    result then rounds differently in one element of 2^8, and by one step; twice that is
    allowed here for the sum of the weights, which differs in the same way."""
    s = Sink(fmt, heads, 2048, 3)  # (no cancellation in the results)
    (a, la), (b, lb) = s.run(sms()), s.run(1)
    a, b = D.host_u16(a[0]).astype(np.int64), D.host_u16(b[0]).astype(np.int64)
    assert np.abs(a - b).max() <= 1
    assert (a != b).mean() <= 2 * 2.0 ** -8
    assert (la[0] - lb[0]).abs().max().item() <= 2.0 ** -16 * (1 + lb.abs().max().item())
