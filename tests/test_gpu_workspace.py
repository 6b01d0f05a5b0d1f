"""A workspace of the caller's is refused unless it is dense, on the call's device and large enough."""
import pytest
import torch

import paged_ref as ref
from head_latent_attention_rmsnorm_gb300 import mla

pytestmark = pytest.mark.gpu


def calls():
    d = mla.dims(4, 64, 32, 16, 32)
    g = ref.generator(1)
    c, k, table = ref.cache(g, d, torch.float32, [5, 9], 4, junk=0.0)
    q, r, w = ref.queries(g, d, torch.float32, 2)
    q, r, c, k, table, w = (x.cuda() for x in (q, r, c, k, table, w))
    lens = torch.tensor([5, 9], dtype=torch.int32, device="cuda")
    x = torch.randn(8, 64, device="cuda")
    return {
        "paged_decode": lambda ws: mla.paged_decode(d, q, r, c, k, table, lens, w, workspace=ws),
        "decode_splitkv": lambda ws: mla.decode_splitkv(d, q, r, c[:2], k[:2], w, workspace=ws),
        "rmsnorm_bwd": lambda ws: mla.rmsnorm_bwd(x, x[0].clone(), x, workspace=ws),
    }


@pytest.mark.parametrize("name", ["paged_decode", "decode_splitkv", "rmsnorm_bwd"])
def test_workspace_refusals(name):
    call = calls()[name]
    room = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    for bad in (room[::2], room[:1].expand(1 << 24), room.view(1 << 12, 1 << 12).t()):
        with pytest.raises(ValueError, match="contiguous"):
            call(bad)
    with pytest.raises(ValueError, match="workspace"):
        call(room.cpu())
    with pytest.raises(ValueError, match="workspace"):
        call(4096)
    with pytest.raises(mla.MlaError, match="WORKSPACE"):
        call(room[:16])
    assert not bool(room.any())
    call(room)
    torch.cuda.synchronize()
