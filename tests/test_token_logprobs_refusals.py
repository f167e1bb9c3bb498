"""Host-side refusals of the token log-probability entry points (CPU)."""

import pytest
import torch

from bit_nf4_quantized_blk_b200 import binding


@pytest.fixture(scope="module")
def lib():
    from bit_nf4_quantized_blk_b200 import build

    build.build()
    return binding.lib()


def test_forward(lib):
    def f(x=16, dtype=0, M=4, V=100, ld=104, t=8, it=1.0, lp=4, H=4, m=4, ls=4, k=3, ids=4, lps=4):
        return lib.qlora_token_logprobs_fwd(x, dtype, M, V, ld, t, it, lp, H, m, ls, k, ids, lps, None)

    ready = (5, 7)  # nothing but the missing device
    assert f() in ready and f(dtype=1) in ready and f(k=32) in ready
    assert f(k=0, ids=None, lps=None) in ready
    assert f(t=None, lp=None) in ready
    assert f(x=None) == 1 and f(dtype=2) == 1 and f(M=0) == 1 and f(V=0) == 1 and f(ld=96) == 1
    assert f(V=1 << 31, ld=1 << 31, M=1) == 7 and f(M=1 << 40) == 7 and f(M=1 << 31, V=8, ld=8) == 7
    assert f(it=0.0) == 1 and f(it=-1.0) == 1 and f(it=float("inf")) == 1 and f(it=float("nan")) == 1
    assert f(it=2.0**100) in ready and f(it=2.0**101) == 1
    assert f(t=None) == 1 and f(lp=None) == 1
    assert f(k=-1) == 1 and f(k=33) == 1 and f(k=5, V=4) == 1 and f(k=0) == 1 and f(ids=None) == 1 and f(lps=None) == 1
    assert f(t=None, lp=None, H=None, m=None, ls=None, k=0, ids=None, lps=None) == 1
    assert f(x=24) == 2 and f(ld=100) == 2 and f(dtype=1, ld=102) == 2
    assert f(dtype=1, ld=100) in ready  # 400-byte rows
    assert f(t=4) == 2 and f(lp=2) == 2 and f(H=2) == 2 and f(m=2) == 2 and f(ls=2) == 2
    assert f(ids=2) == 2 and f(lps=2) == 2


def test_backward(lib):
    def f(x=16, dtype=0, M=4, V=100, ld=104, t=8, it=1.0, m=4, ls=4, H=4, gl=4, gh=4, d=32, ldd=112):
        return lib.qlora_token_logprobs_bwd(x, dtype, M, V, ld, t, it, m, ls, H, gl, gh, d, ldd, None)

    ready = (5, 7)
    assert f() in ready and f(t=None, gl=None) in ready and f(H=None, gh=None) in ready
    assert f(d=16, ldd=104) in ready  # in place
    assert f(d=16) == 1  # in place with another pitch
    assert f(d=None) == 1 and f(ldd=96) == 1 and f(ldd=108) == 2 and f(d=40) == 2
    assert f(x=None) == 1 and f(M=0) == 1 and f(dtype=-1) == 1 and f(it=0.0) == 1
    assert f(m=None) == 1 and f(ls=None) == 1
    assert f(t=None) == 1 and f(gl=None) == 1 and f(H=None) == 1 and f(gh=None) == 1
    assert f(t=None, gl=None, H=None, gh=None) == 1
    assert f(M=1 << 30, V=1 << 9, ld=1 << 9, ldd=1 << 9) in ready
    assert f(M=1 << 30, V=1 << 13, ld=1 << 13, ldd=1 << 13) == 7
    for name in ("m", "ls", "H", "gl", "gh"):
        assert f(**{name: 2}) == 2, name
    assert f(t=4) == 2


def test_binding(monkeypatch):
    x = torch.zeros(4, 104, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int64)
    f32 = torch.zeros(4)
    with pytest.raises(ValueError, match="logits: must be a CUDA tensor"):
        binding.qlora_token_logprobs_fwd(x, t, 1.0, f32, None, None, None, 0, None, None)
    monkeypatch.setattr(binding, "_check_placement", lambda t, name: None)

    def fwd(x=x, t=t, lp=f32, k=0, ids=None, lps=None):
        binding.qlora_token_logprobs_fwd(x, t, 1.0, lp, None, None, None, k, ids, lps)

    with pytest.raises(ValueError, match="2-D"):
        fwd(x=x[0])
    with pytest.raises(TypeError, match="logits: dtype torch.float16"):
        fwd(x=x.half())
    with pytest.raises(ValueError, match="contiguous"):
        fwd(x=torch.zeros(104, 4, dtype=torch.bfloat16).t())
    with pytest.raises(ValueError, match="contiguous"):
        fwd(x=x[:1].expand(4, 104))
    with pytest.raises(TypeError, match="targets: dtype torch.int32"):
        fwd(t=t.int())
    with pytest.raises(ValueError, match="targets: 3 elements, needs at least 4"):
        fwd(t=t[:3])
    with pytest.raises(ValueError, match="top_ids: 4 elements, needs at least 8"):
        fwd(k=2, ids=torch.zeros(4, dtype=torch.int32), lps=torch.zeros(8))
    with pytest.raises(binding.QloraError, match="ALIGNMENT"):
        binding.qlora_token_logprobs_fwd(torch.zeros(4, 101, dtype=torch.bfloat16), t, 1.0, f32, None, None, None, 0,
                                         None, None, stream=0)
    with pytest.raises(ValueError, match="dlogits"):
        binding.qlora_token_logprobs_bwd(x, t, 1.0, f32, f32, None, f32, None, x.float())
    with pytest.raises(ValueError, match="dlogits"):
        binding.qlora_token_logprobs_bwd(x, t, 1.0, f32, f32, None, f32, None, x[:, :96])
