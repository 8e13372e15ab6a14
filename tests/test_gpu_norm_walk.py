"""
The backward's walk over rows: two turns of a row group and more, the last of
them short, at every row shape of the kernels, against f64.
"""

import pytest
import torch

import f8_ref as R
from test_gpu_norm import DT, _f64, _grad_bounds, _grads, _inputs

pytestmark = pytest.mark.gpu


# rows a turn takes at these widths: 2048, 2048, 1024, 512, 512, then 256
@pytest.mark.parametrize("T,D", [(4200, 256), (2100, 1000), (2100, 1024), (2070, 1536), (1030, 2056), (600, 4096),
                                 (261, 8192), (530, 4104), (261, 8200), (515, 9000), (261, 16384)])
@pytest.mark.parametrize("res,blk,dxt,par,post,gate,unit", [
    ("f32", "f32", "f32", "f32", True, "channel", False),
    ("bf16", "bf16", "bf16", "bf16", True, "token", True)])
def test_backward_of_many_rows(T, D, res, blk, dxt, par, post, gate, unit):
    v = _inputs(T, D, res, blk, par, post, gate, unit, seed=T + D + 1)
    v["dx"] = v["dx"].to(DT[dxt]).float()
    got = _grads(v, unit, DT[dxt])
    ref = R.norm_grads(*_f64(v, "r", "u", "w", "p", "g", "dr", "dx"), 0.7, 1e-5, unit)
    bounds = _grad_bounds(v, ref, unit, T, D)
    assert set(got) == set(ref)
    for name, g in got.items():
        want = {"dresidual": DT[res], "dblock": DT[blk]}.get(name, torch.float32)
        b = bounds[name] + R.half_step(want) * (ref[name].abs() + bounds[name]) + R.smallest(want)
        err = (g.cpu().double() - ref[name]).abs()
        assert bool((err <= b).all()), (name, float((err / b).max()))
