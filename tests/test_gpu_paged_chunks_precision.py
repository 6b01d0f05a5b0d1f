"""What the explicit form of a paged step rounds, and nothing more: its results against exact ones, within what follows from
the stated roundings alone.

Scores.  K_nope is fp16, each element off by a uniform rounding of its own, variance u^2 / 12, u its unit in the last place; a
request's first 128 rests keys (rests = min(tokens / 16, 4, its key tiles)) have the rest too and count as exact.  q_nope and the cached
band are bf16, exact in fp16; the rotated q_pe is fp16 with its rest.  So score s_j of key j is off by a variance
w_j = scale^2 sum_d q_d^2 u_jd^2 / 12, independently from key to key.
Log-sum-exp: sum p_j ds_j, a variance sum p_j^2 w_j; its mean square over the rows is near that (the rows' queries are
independent; 1.25 for the sample).  To that come, with a bias, the tensor core's additions, which truncate: a score is 24 of them,
on average half of 2^-23 of a partial sum below |s| + D each (D = sqrt(sum of its squared terms), a walk tied at both ends):
2^-19 (|s| + D) with the sums inside an instruction; K_nope's own 32 shrink it by at most 2^-20: 2^-20 |s|; and exponential, sum,
logarithm and the merge of the two groups: 2^-22 (1 + |lse|).
Outputs: the rounding to bf16, whose relative deviation r is measured on the exact output; P and V in fp16, 2^-4 and 2^-3 of r
(a step eight times as fine; each averages over the keys); the scores' errors by their derivative, a variance
sum_j p_j^2 (v_j - o)^2 w_j; and 1.1 for what the mantissas' spread makes of r."""
import math

import pytest
import torch

import paged_ref as ref
import paged_step_ref as sref
from head_latent_attention_rmsnorm_gb300 import mla

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64


def unit(x):
    """fp16's unit in the last place at x."""
    return torch.exp2(torch.frexp(x.abs().clamp(min=2.0 ** -14)).exponent.to(F64) - 11)


class Case:
    """One request of `new` tokens behind `past`, explicit: what the kernel gave, what is exact, what is allowed."""

    def __init__(self, heads, past, new, deviation, scale=0.0, base=10000.0, key_rows=None):
        d = mla.dims(heads, 512, 128, 64, 128, base)
        d.softmax_scale = scale
        s = sref.step(ref.generator(heads + past + new), d, BF16, [(past, new)], 64)
        s["q_nope"].mul_(deviation)
        s["q_pe"].mul_(deviation)
        a = sref.on_gpu(s)
        self.out, self.lse = (x.to(F64) for x in mla.paged_prefill(d, *a, key_rows=key_rows))
        absorbed = mla.paged_prefill(d, *a, key_rows=0)
        assert mla.mla_check_device_error() == 0 and not torch.equal(absorbed[0].to(F64), self.out)   # (the form)
        n, H = past + new, heads
        scale = scale if scale > 0 else 1.0 / math.sqrt(192)
        rows = (s["block_table"][0, :-(-n // 64)].long()[:, None] * 64 + torch.arange(64)).view(-1)[:n].cuda()
        c, kr = a[2].view(-1, 512)[rows].to(F64), a[3].view(-1, 64)[rows].to(F64)
        w = a[8].to(F64).view(H, 256, 512)
        q = a[0].to(F64)
        pos = s["positions"][:, None].expand(new, H)
        qr = ref.rope(s["q_pe"], pos, base).cuda()
        held = qr.half().to(F64)
        see = torch.arange(n).cuda()[None] <= s["positions"].cuda()[:, None]
        rested = 128 * min(new // 16, 4, -(-n // 128))
        self.exact, self.exact_lse, self.var, self.all_var, self.chain, self.band, self.out_var = [], [], [], [], [], [], []
        for h in range(H):
            k, v = c @ w[h, :128].T, c @ w[h, 128:].T
            x = ((q[:, h] @ k.T + qr[:, h] @ kr.T) * scale).masked_fill(~see, -math.inf)
            lse = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[:, None])
            o = p @ v
            wj = q[:, h].square() @ (unit(k).square() / 12).T * scale * scale
            left = wj.clone()
            left[:, :rested] = 0
            walk = torch.sqrt(q[:, h].square() @ k.square().T + qr[:, h].square() @ kr.square().T) * scale
            size = torch.where(see, x.abs(), 0.0)
            pw = p.square() * left
            self.exact.append(o)
            self.exact_lse.append(lse)
            self.var.append(pw.sum(1))
            self.all_var.append((p.square() * wj).sum(1))
            self.chain.append(2.0 ** -19 * (p * (size + walk)).sum(1) + 2.0 ** -20 * (p * size).sum(1) + 2.0 ** -22 * (1 + lse.abs()))
            self.band.append(scale * (((held - qr)[:, h] @ kr.T) * p).sum(1))
            self.out_var.append(pw @ v.square() - 2 * o * (pw @ v) + o.square() * pw.sum(1, keepdim=True))
        for name in ("exact", "exact_lse", "var", "all_var", "chain", "band", "out_var"):
            setattr(self, name, torch.stack(getattr(self, name), 1))

    def lse_allowed(self):
        return 1.25 * math.sqrt(float(self.var.mean())) + rms(self.chain)


def rms(x):
    return math.sqrt(float(x.square().mean()))


CASES = [   # heads, past, new
    (16, 0, 300), (16, 1700, 300), (16, 8000, 200), (128, 40, 100), (3, 500, 64), (2, 16000, 200),
]


@pytest.mark.parametrize("heads,past,new", CASES)
@pytest.mark.parametrize("deviation,scale,base", [(1, 0.0, 10000.0), (2, 0.0, 10000.0), (4, 0.0, 500.0), (8, 0.0, 10000.0), (1, 0.2, 1e6), (2, 0.01, 100.0)])
def test_rounds_the_stated_parts_only(heads, past, new, deviation, scale, base):
    x = Case(heads, past, new, deviation, scale, base)
    err = x.lse - x.exact_lse
    assert rms(err) <= x.lse_allowed(), (rms(err), x.lse_allowed())
    off = x.out - x.exact
    r2 = (x.exact.to(BF16).to(F64) - x.exact).square().mean()
    allowed = 1.1 * math.sqrt(float(r2) * (1 + 2.0 ** -6 + 2.0 ** -8) + float(x.out_var.mean()))
    assert rms(off) <= allowed, (rms(off), allowed)


def test_a_part_less_would_show():
    """The bounds above are too tight without K_nope's rest or the band's: computed, not run."""
    for heads, past, new in ((16, 0, 300), (3, 500, 64)):
        x = Case(heads, past, new, 1)
        assert rms(x.band) > x.lse_allowed()
        assert math.sqrt(float(x.all_var.mean())) > x.lse_allowed()


@pytest.mark.parametrize("past,new,rel", [(0, 300, 2.5e-7), (1700, 300, 8e-7), (8000, 200, 4e-7)])
def test_documented_figures(past, new, rel):
    """The root mean square error relative to the log-sum-exp at unit scale, as include/mla.h states it (2e-7 to 7e-7)."""
    x = Case(16, past, new, 1)
    assert rms((x.lse - x.exact_lse) / x.exact_lse) <= rel
