"""Host-side refusals of the residual-norm entry points (CPU)."""

import ctypes

import pytest
import torch

from bit_nf4_quantized_blk_b200 import binding


@pytest.fixture(scope="module")
def lib():
    from bit_nf4_quantized_blk_b200 import build

    build.build()
    return binding.lib()


def test_forward(lib):
    def f(h=16, y=16, w_post=16, gate=16, scale=1.0, w_pre=16, eps=1e-5, M=4, D=128, res=0, h_out=16, x=16, ckpt=None,
          r1=4, r2=4):
        c = None if ckpt is None else ctypes.byref(binding.QloraAct8C(*ckpt))
        return lib.qlora_residual_norm_fwd(h, y, w_post, gate, scale, w_pre, eps, M, D, res, h_out, x, c, r1, r2, None)

    ready = (5, 7)  # nothing but the missing device
    assert f() in ready
    assert f(w_post=None, r1=None) in ready and f(gate=None) in ready
    assert f(y=None, w_post=None, gate=None, r1=None) in ready
    assert f(x=None, w_pre=None, r2=None) in ready and f(h_out=None) in ready
    assert f(ckpt=(4, 128, 16, 16, 1)) in ready
    assert f(M=0) == 1 and f(D=0) == 1 and f(D=96) == 1 and f(res=2) == 1
    assert f(D=16384) in ready and f(D=16448) == 7 and f(M=1 << 31) == 7
    assert f(h=None) == 1 and f(h_out=None, x=None, w_pre=None, r2=None) == 1
    assert f(scale=float("inf")) == 1 and f(eps=0.0) == 1 and f(eps=float("nan")) == 1
    assert f(y=None) == 1 and f(y=None, w_post=None, r1=None) == 1
    assert f(w_post=None) == 1  # rstd_post without a norm after the block
    assert f(x=None) == 1 and f(w_pre=None) == 1 and f(x=None, w_pre=None) == 1
    assert f(x=None, w_pre=None, r2=None, ckpt=(4, 128, 16, 16, 1)) == 1
    assert f(ckpt=(3, 128, 16, 16, 1)) == 1 and f(ckpt=(4, 64, 16, 16, 1)) == 1 and f(ckpt=(4, 128, 16, 16, 2)) == 1
    assert f(ckpt=(4, 128, 24, 16, 1)) == 2
    for name in ("h", "y", "w_post", "gate", "w_pre", "h_out", "x"):
        assert f(**{name: 24}) == 2, name
    assert f(r1=2) == 2 and f(r2=2) == 2


def test_backward(lib):
    def f(dh_out=16, dx=16, h_out=16, y=16, w_post=16, gate=16, scale=1.0, w_pre=16, r1=4, r2=4, M=4, D=128, res=0,
          dh=16, dy=16, dw_post=4, dgate=4, dw_pre=4, ws=256, ws_bytes=1 << 30):
        return lib.qlora_residual_norm_bwd(dh_out, dx, h_out, y, w_post, gate, scale, w_pre, r1, r2, M, D, res, dh, dy,
                                           dw_post, dgate, dw_pre, ws, ws_bytes, None)

    ready = (5, 7)
    none = dict(dw_post=None, dgate=None, dw_pre=None)
    assert f() in ready
    assert f(dh_out=None) in ready
    assert f(dx=None, h_out=None, w_pre=None, r2=None, dw_pre=None) in ready
    assert f(**none, ws=None, ws_bytes=0) in ready
    assert f(y=None, w_post=None, gate=None, r1=None, dw_post=None, dgate=None) in ready
    assert f(M=0) == 1 and f(D=100) == 1 and f(res=-1) == 1 and f(D=32768) == 7
    assert f(dh_out=None, dx=None) == 1
    assert f(dh=None, dy=None, **none) == 1
    assert f(scale=float("nan")) == 1
    assert f(h_out=None) == 1 and f(w_pre=None) == 1 and f(r2=None) == 1
    assert f(dx=None) == 1  # dw_pre without dx
    assert f(r1=None) == 1 and f(w_post=None) == 1  # dw_post without its norm
    assert f(gate=None) == 1 and f(y=None) == 1
    for name in ("dh_out", "dx", "h_out", "y", "w_post", "gate", "w_pre", "dh", "dy"):
        assert f(**{name: 24}) == 2, name
    for name in ("r1", "r2", "dw_post", "dgate", "dw_pre"):
        assert f(**{name: 6}) == 2, name
    assert f(ws=None) == 4 and f(ws=128) == 2 and f(ws_bytes=256) == 4
    assert f(ws_bytes=binding.qlora_residual_norm_ws_bytes(4, 128)) in ready


def test_ws_bytes(lib):
    assert binding.qlora_residual_norm_ws_bytes(0, 128) == 0
    assert binding.qlora_residual_norm_ws_bytes(4, 96) == 0
    assert binding.qlora_residual_norm_ws_bytes(4, 1 << 15) == 0
    assert binding.qlora_residual_norm_ws_bytes(4, 128) >= 256 + 2 * 128 * 4


def test_binding(monkeypatch):
    h = torch.zeros(4, 128, dtype=torch.bfloat16)
    w = torch.zeros(128)
    with pytest.raises(ValueError, match="h: must be a CUDA tensor"):
        binding.qlora_residual_norm_fwd(h, None, None, None, 1.0, w, 1e-5, None, h, None, None, None)
    monkeypatch.setattr(binding, "_check_placement", lambda t, name: None)

    def fwd(h=h, y=h, w_post=w, w_pre=w, h_out=h, x=h, ckpt=None):
        binding.qlora_residual_norm_fwd(h, y, w_post, None, 1.0, w_pre, 1e-5, h_out, x, ckpt, None, None)

    with pytest.raises(ValueError, match="2-D"):
        fwd(h=h[0])
    with pytest.raises(TypeError, match="h: dtype torch.float16"):
        fwd(h=h.half())
    with pytest.raises(TypeError, match="h_out: dtype torch.float32"):
        fwd(h_out=h.float())
    with pytest.raises(TypeError, match="w_pre: dtype torch.bfloat16"):
        fwd(w_pre=w.bfloat16())
    with pytest.raises(ValueError, match="y: 384 elements, needs at least 512"):
        fwd(y=h[:3])
    with pytest.raises(ValueError, match="w_post: 64 elements"):
        fwd(w_post=w[:64])
    with pytest.raises(ValueError, match="contiguous"):
        fwd(x=torch.zeros(128, 4, dtype=torch.bfloat16).t())
    with pytest.raises(ValueError, match="gives the shape"):
        binding.qlora_residual_norm_bwd(None, h, None, None, None, None, 1.0, w, None, w, None, h, None, None, None,
                                        None)
    with pytest.raises(TypeError, match="dh: dtype torch.float32"):
        binding.qlora_residual_norm_bwd(h, h, h, None, None, None, 1.0, w, None, w[:4], h.float(), None, None, None,
                                        None, None)
