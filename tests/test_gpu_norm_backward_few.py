"""The norm's backward pass on either side of the sizes where the weight's gradient
is summed beside the rows (1536 rows, 11 2^19 values), in place too.  Bounds as in
test_gpu_norm.py: a lane's chain has at most 12 rows, 4 lanes and 8 to 16 waves."""
from __future__ import annotations

import pytest
import torch

from tests.parity import say
from tests.test_gpu_norm import BF16, F32, backward64, dg, inputs, within  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,h", [(1000, 2111), (1024, 264), (1536, 40), (1537, 40), (1536, 5), (1408, 4096), (1409, 4096),
                                 (804, 7168), (805, 7168), (563, 10240), (564, 10240), (352, 16384), (1300, 1161)])
@pytest.mark.parametrize("weight", [F32, BF16])
def test_backward(dg, t, h, weight):  # noqa: F811
    say(f"norm backward {t}x{h} weight={weight}")
    few = t <= 1536 and t * h <= 11 << 19
    assert (dg.rmsnorm_bf16_backward_workspace(t, h) == 0) == few
    dy, ds, w = inputs(t, h, True, weight, 41)
    z = inputs(t, h, False, None, 42)[0]
    rstd = torch.rsqrt(z.float().square().mean(1) + 1e-6)
    dx, dw = torch.full((t, h), float("nan"), dtype=BF16, device="cuda"), torch.full((h,), float("nan"), device="cuda")
    dg.rmsnorm_bf16_backward(dy, z, w, rstd, dx, dw, ds)
    wx, bx, ww, bw = backward64(dy, z, w, rstd, ds)
    within(dx, wx, bx, "dx")
    within(dw, ww, bw, "dw")
    for over in (dy, z, ds):
        args = dict(dy=dy, z=z, ds=ds)
        name = [n for n, v in args.items() if v is over][0]
        args[name] = over.clone()
        two = torch.empty_like(dw)
        dg.rmsnorm_bf16_backward(args["dy"], args["z"], w, rstd, args[name], two, args["ds"])
        assert torch.equal(args[name], dx) and torch.equal(two, dw), name
