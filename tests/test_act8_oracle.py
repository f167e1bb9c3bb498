"""The checkpoint oracle against its definition, and the host-side refusals of
the checkpoint entry points (CPU)."""

import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

from bit_nf4_quantized_blk_b200 import binding
from oracle import act8


@pytest.fixture(scope="module")
def lib():
    from bit_nf4_quantized_blk_b200 import build

    build.build()
    return binding.lib()


@pytest.fixture
def any_device(monkeypatch):
    monkeypatch.setattr(binding, "_check_placement", lambda t, name: None)


def _bf16(v) -> np.ndarray:
    return torch.tensor(v, dtype=torch.float64).to(torch.bfloat16).double().numpy()


def test_round_bf16_matches_torch():
    g = torch.Generator().manual_seed(0)
    v = torch.randn(20000, generator=g, dtype=torch.float64) * torch.exp2(
        torch.randint(-140, 128, (20000,), generator=g).double())
    v = v.float()  # exact fp32 values, so torch's conversion rounds once
    got = act8.round_bf16(v.double().numpy())
    assert np.array_equal(got, v.to(torch.bfloat16).double().numpy())


def test_int8_codes_are_the_nearest_integers():
    """Against exact rational arithmetic, ties to even, on every pair of significands of one binade."""
    sig = [Fraction(128 + i, 128) for i in range(0, 128, 5)]
    for top in sig:
        for scale in (1, Fraction(1, 2), Fraction(1, 16)):
            x = np.zeros(64)
            x[0] = float(top)
            others = [s * scale for s in sig if s * scale <= top][:63]
            x[1:1 + len(others)] = [float(o) for o in others]
            codes, step = act8.encode(x, "int8")
            s = Fraction(float(step[0]))
            for i, o in enumerate([top, *others]):
                assert codes.view(np.int8)[i] == max(-127, min(127, round(o / s))), (top, o)


def test_edges():
    for fmt in ("int8", "e4m3"):
        z = np.zeros(64)
        codes, step = act8.encode(z, fmt)
        assert step[0] == 0 and not codes.any()
        for bad in (np.nan, np.inf, -np.inf):
            x = np.ones(128)
            x[70] = bad
            codes, step = act8.encode(x, fmt)
            assert np.isnan(step[1]) and step[0] > 0
            v = act8.decode(codes, step, fmt)
            assert np.isnan(v[64:]).all() and np.isfinite(v[:64]).all()
        largest = float(torch.finfo(torch.bfloat16).max)
        x = np.full(64, largest)
        v = act8.decode(*act8.encode(x, fmt), fmt)
        assert np.isfinite(v).all() and (v >= 0.98 * largest).all()


@pytest.mark.parametrize("fmt, rel", [("int8", None), ("e4m3", 2.0**-4 + 2.0**-8)])
def test_reconstruction_error(fmt, rel):
    """int8: half a step and half a bf16 rounding; E4M3: half a step of 3 mantissa bits (or of its smallest)."""
    x = _bf16(np.random.RandomState(1).randn(64 * 200) * 3)
    codes, step = act8.encode(x, fmt)
    err = np.abs(act8.decode(codes, step, fmt) - x)
    s = np.repeat(step, 64)
    if fmt == "int8":
        assert (err <= 0.5 * s + 2.0**-8 * (np.abs(x) + 0.5 * s)).all()
    else:
        assert (err <= np.maximum(rel * np.abs(x), 2.0**-10 * s * (1 + 2.0**-7))).all()


def test_library_refusals(lib):
    """Every check runs on the host before anything is enqueued (no device here)."""
    C = binding.QloraAct8C
    ok = (4, 128, 16, 16, 0)

    def q(a, x=16):
        return lib.qlora_act8_quantize(x, ctypes.byref(C(*a)), None)

    def d(a, x=16):
        return lib.qlora_act8_dequantize(ctypes.byref(C(*a)), x, None)

    for f in (q, d):
        assert f(ok) in (5, 7)  # nothing but the missing device
        assert f((0, 128, 16, 16, 0)) == 1
        assert f((4, 0, 16, 16, 0)) == 1
        assert f((4, 96, 16, 16, 0)) == 1
        assert f((4, 128, None, 16, 0)) == 1
        assert f((4, 128, 16, None, 0)) == 1
        assert f((4, 128, 16, 16, 2)) == 1
        assert f((4, 128, 16, 16, -1)) == 1
        assert f((4, 128, 24, 16, 0)) == 2
        assert f((4, 128, 16, 17, 0)) == 2
        assert f((1 << 40, 128, 16, 16, 0)) == 7
        assert f(ok, None) == 1
        assert f(ok, 24) == 2
    assert lib.qlora_act8_quantize(16, None, None) == 1
    assert lib.qlora_act8_dequantize(None, 16, None) == 1

    W = binding.QloraNf4WeightC(64, 128, 16, 16, 16, 16)

    def b(a=ok, w=W, r=8, dY=16, acc=0, ws=256, ws_bytes=1 << 30, A=16, U=None, scale=1.0):
        return lib.qlora_linear_bwd_act8(ctypes.byref(w), ctypes.byref(C(*a)) if a else None, dY, A, 16, r, scale, U,
                                         None, acc, None, None, ws, ws_bytes, None)

    assert b() in (5, 7)
    assert b(a=None) == 1
    assert b(a=(4, 64, 16, 16, 0)) == 1  # the checkpoint's columns are not the weight's
    assert b(a=(0, 128, 16, 16, 0)) == 1
    assert b(a=(4, 128, 16, 16, 3)) == 1
    assert b(r=0) == 1 and b(r=65) == 1
    assert b(dY=None) == 1 and b(A=None) == 1
    assert b(acc=2) == 1
    assert b(scale=float("nan")) == 1
    assert b(dY=24) == 2 and b(U=18) == 2
    assert b(ws=None) == 4 and b(ws_bytes=256) == 4
    assert b(w=binding.QloraNf4WeightC(64, 128, None, 16, 16, 16)) == 1


def test_binding_refusals(any_device):
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    a = binding.Act8.empty(4, 128, device="cpu")
    for rows, cols in ((0, 128), (4, 0), (4, 96)):
        with pytest.raises(ValueError, match="multiple of 64"):
            binding.Act8.empty(rows, cols, device="cpu")
    with pytest.raises(TypeError, match="X: dtype"):
        binding.qlora_act8_quantize(x.float(), a)
    with pytest.raises(ValueError, match="X: 256 elements, needs at least 512"):
        binding.qlora_act8_quantize(x[:2], a)
    with pytest.raises(ValueError, match="contiguous"):
        binding.qlora_act8_dequantize(a, torch.zeros(128, 4, dtype=torch.bfloat16).t())
    short = binding.Act8(4, 128, a.codes[:3], a.step, binding.ACT8_INT8)
    with pytest.raises(ValueError, match="codes: 384 elements"):
        binding.qlora_act8_dequantize(short, x)
    wrong = binding.Act8(4, 128, a.codes, a.step.float(), binding.ACT8_INT8)
    with pytest.raises(TypeError, match="step: dtype"):
        binding.qlora_act8_dequantize(wrong, x)
    w = binding.NF4Weight.empty(8, 128, device="cpu")
    A, B = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(8, 4, dtype=torch.bfloat16)
    ws = torch.empty(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="dY: 8 elements, needs at least 32"):
        binding.qlora_linear_bwd_act8(w, a, torch.zeros(1, 8, dtype=torch.bfloat16), A, B, 4, 1.0, None, 0, None,
                                      None, ws)


def test_cpu_tensors_are_refused():
    a = binding.Act8.empty(4, 128, device="cpu")
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.qlora_act8_quantize(torch.zeros(4, 128, dtype=torch.bfloat16), a)
