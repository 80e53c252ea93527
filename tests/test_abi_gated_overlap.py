"""Refusals of the gated layer: one buffer given for two, where one would be overwritten while it is still
read, or by the other, and an empty list.  All before anything is enqueued."""
import os

import pytest
import torch

import grouped_gemm_gl_amd as gl
from test_abi_gated import A, B, C_, GLU, GLU_B, INT8

pytestmark = pytest.mark.skipif(not os.path.exists(gl.library_path), reason="library not built")
H = 0x700000  # another aligned address, never dereferenced


@pytest.mark.parametrize("kw", [dict(a=A), dict(h=A)], ids=str)  # a or h in x's place
def test_forward(kw):
    assert gl.load().gl_glu_forward(*{**GLU, **kw}.values(), None) == -1 and gl.load().gl_last_error()


@pytest.mark.parametrize("kw", [
    dict(h=H, a=H),           # a over the kept h, which other threads still read
    dict(dh=A, dw=H),         # dh over x, which dW is the product of
    dict(a=A, dw=H),          # a over x
    dict(dx=GLU_B["dh"]),     # dx over dh, while other rows' products read it
    dict(a=H, dx=H),          # two outputs
], ids=str)
def test_backward(kw):
    assert gl.load().gl_glu_backward(*{**GLU_B, **kw}.values(), None) == -1 and gl.load().gl_last_error()


def test_int8_products():
    v = list({**INT8, "y": INT8["x"]}.values())
    assert gl.load().gl_forward_int8(*v, None) == -1 and gl.load().gl_last_error()
    assert gl.load().gl_glu_forward_int8(*v[:5], 0, *v[5:], None) == -1 and gl.load().gl_last_error()


def test_backward_refuses_an_empty_list_of_gradients():
    t = lambda *s: torch.empty(*s)  # noqa: E731
    with pytest.raises(ValueError, match="dw"):
        gl.gl_glu_backward(t(3, 64), t(2, 32, 64), t(3, 16), t(3, 32), None, [], torch.empty(gl.gl_workspace_size(2), dtype=torch.uint8))
