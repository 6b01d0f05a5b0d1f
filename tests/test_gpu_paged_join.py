"""The last launch of a step's absorbed form where its blocks find few tokens or none: a list shorter than the grid,
turns and whole steps of rows that belong to no request.  Such steps run one behind another, so that what a block left
behind would reach the next one's shared memory."""
import pytest
import torch

import paged_ref as ref
import paged_step_ref as sref
from head_latent_attention_rmsnorm_gb300 import mla

pytestmark = pytest.mark.gpu

V3 = dict(d_kv=512, d_nope=128, d_rope=64, d_v=128)
BF = torch.bfloat16


@pytest.mark.parametrize("heads", [4, 16, 64])
@pytest.mark.parametrize("lens,lead,extra", [
    ([(0, 300), (40, 2)], 0, 0),        # two tokens in a list of 302
    ([(0, 290), (400, 33)], 0, 0),      # a block of one token
    ([(30, 3)], 200, 90),               # turns of rows of no request around one of three
    ([(30, 0), (0, 0)], 130, 0),        # nothing but such rows
])
def test_blocks_without_a_token(heads, lens, lead, extra):
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(heads), d, BF, lens, 16, extra_rows=extra, lead=lead)
    a = sref.on_gpu(s)
    n = s["positions"].numel()
    before = (torch.full((n, heads, 128), 5.0, dtype=BF).cuda(), torch.full((n, heads), 6.0).cuda())
    for key_rows in (None, 0):
        ws = mla.paged_prefill_workspace(d, n, a[2], a[4], key_rows=key_rows)
        outs = [tuple(x.clone() for x in before) for _ in range(20)]
        for out, lse in outs:
            mla.paged_prefill(d, *a, key_rows=key_rows, out=out, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        assert mla.mla_check_device_error(None) == 0
        for out, lse in outs[1:]:
            assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])
        own = torch.tensor(sref.owners(s))
        out, lse = outs[0]
        assert torch.equal(out.cpu()[own < 0], before[0].cpu()[own < 0]) and torch.equal(lse.cpu()[own < 0], before[1].cpu()[own < 0])
        few = [t for t, b in enumerate(own.tolist()) if b >= 0][-3:]
        if few:
            rows = dict(s, q_nope=s["q_nope"][few], q_pe=s["q_pe"][few], positions=s["positions"][few],
                        block_table=s["block_table"][own[few]], kv_lens=s["kv_lens"][own[few]],
                        cu_tokens=torch.arange(len(few) + 1, dtype=torch.int32))
            ref.check_decode(BF, out[few].cpu(), lse[few].cpu(), sref.prefill(d, rows))
