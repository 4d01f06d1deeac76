"""GPU: what the binding of the 4-bit calls refuses on the host because a kernel would read it on the device."""
import pytest
import torch

import combine_router_gemm_amd as moe
from tests.test_gpu_w4 import DEV, case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["expert_kept", "expert_offset"])
@pytest.mark.parametrize("change", ["host", "type", "short", "strided"])
def test_layout_arrays(name, change):
    """Each array of the layout that the expert MLP reads: on the host, of another type, too short, not contiguous."""
    L, send, packs, _ = case([3, 2, 0, 1], 6, 1, 1, 6, 32, 32, 3)
    out = torch.full((L.rows_max, 32), -7.0, dtype=torch.bfloat16, device=DEV)
    good = getattr(L, name)
    setattr(L, name, {"host": good.cpu(), "type": good.long(), "short": good[:-1].clone(),
                      "strided": good.repeat_interleave(2)[::2]}[change])
    with pytest.raises(moe.MoeError, match=name):
        moe.moe_expert_mlp_w4(send.to(DEV), L, *packs, out)
    assert torch.all(out == -7.0)
    setattr(L, name, good)
    moe.moe_expert_mlp_w4(send.to(DEV), L, *packs, out)
    assert torch.all(out != -7.0)
