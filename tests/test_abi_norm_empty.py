"""
Norm calls of no rows through the C ABI, on the host: tensors without rows have
no pointer, and no call may need one. (The backward also writes its parameters'
gradients, on the GPU: test_gpu_views.py.)
"""

import pytest

import mixture_experts_routed_route_amd as moe
from test_abi_f8 import _back, _desc, _norm


@pytest.mark.parametrize("kind", [moe.MOE_GATE_NONE, moe.MOE_GATE_CHANNEL, moe.MOE_GATE_TOKEN])
@pytest.mark.parametrize("post,pre", [(0x3000, 0x4000), (None, 0x4000), (0x3000, None), (None, None)])
def test_forward_of_no_rows(post, pre, kind):
    gate = 0xB000 if kind == moe.MOE_GATE_CHANNEL else None
    d = _desc(T=0, gate_kind=kind)
    assert _norm(moe.library(), d, r=None, u=None, p=post, g=gate, w=pre, ro=None, x=None) == moe.MOE_OK


def test_backward_still_refuses():
    L, E = moe.library(), moe.MOE_EINVAL
    empty = dict(r=None, u=None, dro=None, dx=None, dr=None, du=None)
    assert _back(L, _desc(T=0), **dict(empty, dw=None)) == E
    assert _back(L, _desc(T=0), **dict(empty, dp=None)) == E
    assert _back(L, _desc(T=0, gate_kind=moe.MOE_GATE_CHANNEL), **empty) == E
    assert _back(L, _desc(T=0), **dict(empty, work=None)) == E
    # the workspace is asked for after every pointer
    for kind in (moe.MOE_GATE_NONE, moe.MOE_GATE_TOKEN):
        assert _back(L, _desc(T=0, gate_kind=kind), nbytes=0, **empty) == moe.MOE_EWORKSPACE
