"""What the tensor-core paged decode rounds, and nothing more: its results against a 64-bit model that takes exactly
the stated parts of the queries in the scores, on both sides of every length and head count where those change.

The model.  The absorbed query q = W_K^T q_nope is held as bf16 parts hi + lo (+ rest); the scores take q_hi and q_lo of
the blocks of 64 latent dims that `parts` names, the rest of q_lo shifts the log-sum-exp by scale q_lo . o, and up
to 64 keys so does q_rest.  Everything else is exact.  What then parts the kernel from the model:
* the output's rounding to bf16, whose relative deviation r is measured on the exact output;
* above 64 heads P's rounding to bf16: each weight is off by a rounding like the output's, independently, so the
  sum over the keys by the same r of sqrt(sum p^2 c^2) <= |o|;
* fp16 partial sums, 2^-3 of r; fp32 arithmetic, 2^-12 of r.
Hence an error of at most r (1 + 2^-6)^(1/2), or r (2 + 2^-6)^(1/2), and 1.1 for what the mantissas' spread makes of r.
The log-sum-exp: a score is a chain of at most 48 fp32 additions, each off by at most 2^-23 of the partial sum if the
tensor core truncates, half of that on average.  A chain of terms t_d that ends at s has partial sums of i/N s on average
with a deviation of at most D / 2, D = sqrt(sum t_d^2) (a walk tied at both ends), so of a size below |s| + D: the mean
over the weights is off by 24 * 2^-23 E(|s| + D) < 2^-18 E(|s| + D).  (D is 1 at unit scale and grows with the queries'; a
single key whose score happens to be near zero has it all the same.)  2^-21 |lse| covers exp, sum, log and the merge."""
import math

import pytest
import torch

import paged_ref as ref
from head_latent_attention_rmsnorm_gb300 import mla

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64
BLOCKS = 8


def parts(heads, keys):
    """Blocks of 64 latent dims whose q_lo the scores take."""
    if heads <= 64:
        return range(BLOCKS)
    return (1, 2, 3) if keys <= 64 else range(4) if keys <= 1024 else range(2) if keys <= 4096 else ()


def model(d, q_nope, q_pe, c, k, w, n, taken):
    """One request of n keys: (out, lse, E(|s| + D)) with q_lo of the blocks `taken` in the scores; None: of no rounding."""
    H, dn, dk = d.n_heads, d.d_nope, d.d_kv
    scale = 1.0 / math.sqrt(dn + d.d_rope)
    w = w.to(F64).view(H, dn + d.d_v, dk)
    q = torch.matmul(q_nope.to(F64)[:, None], w[:, :dn])[:, 0]
    qr = ref.rope(q_pe.cpu(), torch.full((H,), n - 1), d.rope_base).to(c.device)
    held = q
    if taken is not None:
        hi = q.float().to(BF16).to(F64)
        lo = (q - hi).float().to(BF16).to(F64)
        keep = torch.zeros(dk, dtype=F64, device=c.device)
        for b in taken:
            keep[64 * b:64 * b + 64] = 1
        held = hi + lo * keep
    c, k = c.to(F64), k.to(F64)
    s = (held @ c.T + qr @ k.T) * scale
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    o = p @ c
    if taken is not None:
        left = lo * (1 - keep) + (q - hi - lo if n <= 64 else 0)
        lse = lse + scale * (left * o).sum(1)
    walk = torch.sqrt(held.square() @ c.square().T + qr.square() @ k.square().T) * scale
    return torch.matmul(w[:, dn:], o[:, :, None])[:, :, 0], lse, (p * (s.abs() + walk)).sum(1)


def case(heads, keys, deviation, page=64):
    d = mla.dims(heads, 512, 128, 64, 128)
    g = ref.generator(heads + keys)
    B = max(2, 128 // heads)
    lens = [keys] * B
    c, k, table = ref.cache(g, d, BF16, lens, page)
    q, r, w = ref.queries(g, d, BF16, B)
    q, r = (q * deviation).to(BF16), (r * deviation).to(BF16)
    dev = [x.cuda() for x in (q, r, c, k, table, torch.tensor(lens, dtype=torch.int32), w)]
    out, lse = mla.paged_decode(d, *dev)
    assert mla.last_path() == mla.PATH_TC and mla.mla_check_device_error() == 0
    rows = [(table[b, :-(-keys // page)].long()[:, None] * page + torch.arange(page)).view(-1)[:keys].cuda() for b in range(B)]

    def want(taken):
        got = [model(d, dev[0][b], dev[1][b], dev[2].view(-1, 512)[rows[b]], dev[3].view(-1, 64)[rows[b]], dev[6], keys, taken)
               for b in range(B)]
        return [torch.stack(x) for x in zip(*got)]
    return out.to(F64), lse.to(F64), want


def off(a, b):
    return float((a - b).norm() / b.norm())


@pytest.mark.parametrize("deviation", [1, 4, 8])
@pytest.mark.parametrize("keys", [1, 64, 65, 1024, 1025, 4096, 4097])
@pytest.mark.parametrize("heads", [16, 64, 65, 128, 130])
def test_rounds_the_stated_parts_only(heads, keys, deviation):
    out, lse, want = case(heads, keys, deviation)
    taken = parts(heads, keys)
    exact, near = want(None)[0], want(taken)
    r = off(exact.to(BF16).to(F64), exact)
    own = math.sqrt((1 if heads <= 64 else 2) + 2.0 ** -6)
    assert float((out - near[0]).norm() / exact.norm()) <= 1.1 * own * r
    err, bound = (lse - near[1]).abs(), 2.0 ** -18 * near[2] + 2.0 ** -21 * near[1].abs()
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("heads,keys,less", [(16, 64, ()), (16, 65, ()), (64, 1024, ()), (64, 4097, range(7)), (128, 1024, range(2)),
                                             (128, 4096, ()), (130, 1025, ()), (65, 1000, ())])
def test_a_part_less_would_show(heads, keys, less):
    """The bound above is too tight for a decode whose scores took only the parts `less`: computed, not run."""
    out, lse, want = case(heads, keys, 8)
    exact, near, worse = want(None)[0], want(parts(heads, keys)), want(less)
    r = off(exact.to(BF16).to(F64), exact)
    own = math.sqrt((1 if heads <= 64 else 2) + 2.0 ** -6)
    # such a decode has its own roundings, independent of the parts' error, on top
    gone = float((worse[0] - near[0]).norm() / exact.norm())
    assert math.hypot(gone, own * r / 1.1) > 1.1 * own * r


@pytest.mark.parametrize("heads,most", [(16, 1.1), (64, 1.1), (128, 1.1 * math.sqrt(2 + 2 / 3))])
@pytest.mark.parametrize("keys", [65, 1000, 5000])
def test_output_error_at_unit_scale(heads, keys, most):
    """Against exact results, over the rounding's own: 1 up to 64 heads; above, the weights' rounding adds its square
    and q_lo's that of the latent scores' deviation, 2/3 at unit scale."""
    out, _, want = case(heads, keys, 1)
    exact = want(None)[0]
    assert off(out, exact) <= most * off(exact.to(BF16).to(F64), exact)
