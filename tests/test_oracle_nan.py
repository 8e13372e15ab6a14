"""The oracle's expert keeps a NaN of either product through the clamps, as the
numpy brute force and the kernels do."""

import numpy as np
import pytest

import oracle
import workloads as W
from oracle import brute


@pytest.mark.parametrize("which", ["w_gate", "w_up", "x"])
@pytest.mark.parametrize("c", [7.0, 0.0])
def test_expert_keeps_nan(which, c):
    wl = W.make_layer(1, 16, 24, 1, 1, W.F32, seed=5, w_std=0.3)
    if which == "x":
        wl["x"][0, 3] = float("nan")
    else:
        wl[which][0, 5, 3] = float("nan")
    ws = [wl[n] for n in ("w_gate", "w_up", "w_down")]
    h, y = oracle.expert(wl["x"][0], 0, *ws, "f32", "f32", c)[2:]
    assert np.isnan(y).all()
    assert np.isnan(h).all() if which == "x" else np.flatnonzero(np.isnan(h)).tolist() == [5]
    assert np.isnan(brute.expert_dense(wl["x"].numpy().astype(np.float64),
                                       *(w[0].numpy().astype(np.float64) for w in ws), c)).all()
