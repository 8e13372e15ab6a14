"""4-bit groups that hold an infinity or a NaN, or whose scale passes fp16's range,
stand for NaN: every value of them, and every product with them."""

import math

import pytest
import torch

import mixture_experts_routed_route_amd as moe
from q4_ref import DT, FORMATS, GROUP, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_such_groups_stand_for_nan(fmt, dt):
    G = GROUP[fmt]
    step = torch.arange(G).float() - G // 2
    at = lambda v: torch.where(step == 3, v, step)
    rows = [at(math.inf), at(-math.inf), at(math.nan), torch.full((G,), math.inf), torch.full((G,), -math.inf),
            torch.where(step < 0, -math.inf, math.inf), torch.full((G,), math.nan)]
    if dt != "f16":     # finite values whose scale is past 65504
        rows += [step * 1e6, step * 1e36, torch.where(step == 3, 2e6, 0.0)]
    v = torch.stack(rows).to(DT[dt])
    n = v.shape[0]
    v = torch.cat([step.expand(n, G).to(DT[dt]), v, step.expand(n, G).to(DT[dt])], 1).cuda()
    w = moe.moe_quant_q4_weights(v, FORMATS[fmt])
    got = values(w, fmt).unflatten(-1, (3, G))
    assert got[:, 1].isnan().all() and got[:, ::2].isfinite().all()
    deq = moe.moe_dequant_weights(*w).unflatten(-1, (3, G))
    assert deq[:, 1].isnan().all() and torch.equal(deq[:, ::2], got[:, ::2].half())
    x = torch.ones(2, 3 * G, dtype=torch.float16, device="cuda")
    assert moe.moe_gemm_q4(x, w, out_dtype=torch.float32).isnan().all()
