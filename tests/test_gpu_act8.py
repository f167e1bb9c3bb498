"""GPU: 8-bit activation checkpoints, bit for bit against the fp64 oracle, and
the linear backward from them."""

import numpy as np
import pytest
import torch

from bit_nf4_quantized_blk_b200 import binding, workloads
from gpu_helpers import gpu_quantize, require_gpu, workspace
from oracle import act8, lora, nf4

pytestmark = pytest.mark.gpu

FORMATS = {"int8": binding.ACT8_INT8, "e4m3": binding.ACT8_E4M3}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _inputs(M, K, seed, wide=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g)
    if wide:  # every exponent a block can have, and blocks of mixed ones
        x *= torch.exp2(torch.randint(-133, 127, (M, K // 64), generator=g).float()).repeat_interleave(64, 1)
        x[:, ::3] *= 2.0**-7
    x = x.to(torch.bfloat16)
    if M > 2:
        x[M // 2] = 0.0
        x[M // 2, 5::7] = -0.0
    return x


def _check_bits(x, fmt):
    M, K = x.shape
    guard = 64
    a = binding.Act8(M, K, torch.full((M * K + guard,), 0xA5, dtype=torch.uint8, device="cuda"),
                     torch.full((M * K // 64 + guard,), 7.0, dtype=torch.bfloat16, device="cuda"), FORMATS[fmt])
    back = torch.full((M * K + guard,), 9.0, dtype=torch.bfloat16, device="cuda")
    binding.qlora_act8_quantize(x.cuda(), a)
    binding.qlora_act8_dequantize(a, back)
    codes, step = act8.encode(_f64(x), fmt)
    got_step = _f64(a.step)
    assert np.array_equal(got_step[:-guard], step, equal_nan=True)
    assert np.array_equal(a.codes.cpu().numpy()[:-guard], codes)
    want = act8.decode(codes, step, fmt)
    assert np.array_equal(_f64(back)[:-guard], want, equal_nan=True)
    # nothing behind the end is touched
    assert (a.codes[-guard:] == 0xA5).all() and (got_step[-guard:] == 7.0).all() and (back[-guard:] == 9.0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M, K", [(1, 64), (1, 4096), (3, 192), (17, 2048), (129, 1088), (1000, 320)])
def test_codes_and_values(M, K, fmt):
    _check_bits(_inputs(M, K, M + K), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_magnitude(fmt):
    """Blocks from the subnormals to the largest finite values."""
    _check_bits(_inputs(600, 256, 5, wide=True), fmt)
    x = torch.full((3, 64), torch.finfo(torch.bfloat16).max, dtype=torch.bfloat16)
    x[1, ::2] *= -0.5
    x[2] = 2.0**-133
    _check_bits(x, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_ties(fmt):
    """Quotients that lie exactly between two codes: x an odd multiple of half a step, every significand of the step."""
    sig = torch.arange(128, 256).double() / 128
    k = torch.arange(1, 64).double()
    step = sig if fmt == "int8" else sig / 2
    x = torch.zeros(128, 64, dtype=torch.float64)
    x[:, 0] = step * (127 if fmt == "int8" else 256)
    x[:, 1:] = step[:, None] * (k + 0.5) if fmt == "int8" else step[:, None] * (8 + (k % 8) + 0.5)
    _check_bits(x.to(torch.bfloat16), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_nonfinite_blocks(fmt):
    x = _inputs(6, 192, 3)
    x[1, 70] = float("nan")
    x[2, 0] = float("inf")
    x[4, 191] = float("-inf")
    _check_bits(x, fmt)


def _linear(M, N, K, r, seed):
    W = workloads.normal_f32((N, K), 0.02, seed)
    A = workloads.normal_bf16((r, K), 0.05, seed + 1)
    B = workloads.normal_bf16((N, r), 0.05, seed + 2)
    dY = workloads.normal_bf16((M, N), 1.0, seed + 3)
    return W, A, B, dY, _inputs(M, K, seed + 4)


def _checkpoint(x, fmt):
    a = binding.Act8.empty(*x.shape, fmt=FORMATS[fmt])
    binding.qlora_act8_quantize(x.cuda(), a)
    return a


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M, N, K, r", [(1, 64, 64, 1), (16, 72, 128, 5), (17, 136, 192, 8), (33, 40, 4160, 24),
                                        (130, 64, 1088, 16), (300, 72, 576, 33), (257, 128, 1536, 48),
                                        (1000, 256, 2048, 64), (2050, 64, 64, 12), (700, 8, 64, 64),
                                        (1500, 1032, 2112, 40)])
@pytest.mark.parametrize("saved_u", [True, False])
def test_linear_backward(M, N, K, r, fmt, saved_u):
    s = 2.0
    W, A, B, dY, x = _linear(M, N, K, r, M + N + K + r)
    w = gpu_quantize(W)
    a = _checkpoint(x, fmt)
    Ac, Bc, dYc = A.cuda(), B.cuda(), dY.cuda()
    ws = workspace(M, N, K, r)
    codes, step = act8.encode(_f64(x), fmt)
    xh = act8.decode(codes, step, fmt).reshape(M, K)
    U = torch.from_numpy((_f64(x) @ _f64(A).T).astype(np.float32)).cuda() if saved_u else None
    dX = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    dA = torch.full((r + 1, K), 3.0, dtype=torch.float32, device="cuda")
    dB = torch.full((N + 1, r), 3.0, dtype=torch.float32, device="cuda")
    binding.qlora_linear_bwd_act8(w, a, dYc, Ac, Bc, r, s, dX, 0, dA, dB, ws, U=U)
    assert binding.qlora_workspace_status(ws) == 0
    assert (dA[r] == 3.0).all() and (dB[N] == 3.0).all()

    g, b64 = _f64(dY), _f64(B)
    u = U.double().cpu().numpy() if saved_u else xh @ _f64(A).T
    # V and U enter as three bf16 parts, which hold all of their fp32 values; V itself is an fp32 sum of N products, and
    # each output one of 3 M: at most (terms) 2^-24 of the sum of magnitudes each.
    absv = np.abs(g) @ np.abs(b64)
    ref = s * (g @ b64).T @ xh
    tol = (N + 3 * M + 2) * 2.0**-24 * s * absv.T @ np.abs(xh) + 1e-30
    assert (np.abs(_f64(dA[:r]) - ref) <= tol).all()
    absu = np.abs(u) if saved_u else np.abs(xh) @ np.abs(_f64(A)).T
    ref = s * g.T @ u
    tol = (3 * M + 2 + (0 if saved_u else K)) * 2.0**-24 * s * np.abs(g).T @ absu + 1e-30
    assert (np.abs(_f64(dB[:N]) - ref) <= tol).all()

    # dX does not depend on X.  Ranks up to 16 share V's kernel with the bf16 path: the same bits.  Above, V is summed in
    # another order: both are within e = N 2^-24 sum |dY| |B| of the exact V, so their bf16 roundings (2^-8 each) differ
    # by at most 2^-7 (|V| + e) + 2 e; and dX is rounded once on each side.
    dX2 = torch.empty_like(dX)
    dA2, dB2 = torch.empty((r, K), device="cuda"), torch.empty((N, r), device="cuda")
    binding.qlora_linear_bwd(w, x.cuda(), dYc, Ac, Bc, r, s, dX2, 0, dA2, dB2, ws, U=U)
    if r <= 16 and M > 16:
        assert torch.equal(dX, dX2)
    else:
        e = N * 2.0**-24 * absv
        apart = s * (2.0**-7 * (np.abs(g @ b64) + e) + 2 * e) @ np.abs(_f64(A))
        assert (np.abs(_f64(dX) - _f64(dX2)) <= apart + 2.0**-7 * np.abs(_f64(dX)) + 1e-30).all()
    if saved_u:  # the bf16 path splits U in two parts
        assert (dB[:N] - dB2).norm() <= 4e-6 * dB2.norm()


def test_linear_backward_agrees_with_the_dequantized_activation():
    """qlora_linear_bwd on the checkpoint's bf16 values is the same product, from V and U in two bf16 parts (2^-17 at
    most) and summed in another order."""
    M, N, K, r = 700, 192, 1024, 16
    W, A, B, dY, x = _linear(M, N, K, r, 77)
    w, ws = gpu_quantize(W), workspace(M, N, K, r)
    for fmt in FORMATS:
        a = _checkpoint(x, fmt)
        xb = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
        binding.qlora_act8_dequantize(a, xb)
        outs = []
        for call, X in ((binding.qlora_linear_bwd_act8, a), (binding.qlora_linear_bwd, xb)):
            dA, dB = torch.empty((r, K), device="cuda"), torch.empty((N, r), device="cuda")
            call(w, X, dY.cuda(), A.cuda(), B.cuda(), r, 1.0, None, 0, dA, dB, ws)
            outs.append((dA, dB))
        for p, q in zip(*outs):
            assert (p - q).norm() <= 2.0**-17 * q.norm()


@pytest.mark.parametrize("fmt", FORMATS)
def test_linear_backward_variants(fmt):
    """Accumulation into dX, outputs left out, and a dense-weight path."""
    M, N, K, r = 65, 128, 320, 8
    W, A, B, dY, x = _linear(M, N, K, r, 5)
    w, a = gpu_quantize(W), _checkpoint(x, fmt)
    Ac, Bc, dYc = A.cuda(), B.cuda(), dY.cuda()
    ws = workspace(M, N, K, r)

    def run(dX=None, acc=0, da=True, db=True, ws=ws):
        dA = torch.empty((r, K), device="cuda") if da else None
        dB = torch.empty((N, r), device="cuda") if db else None
        binding.qlora_linear_bwd_act8(w, a, dYc, Ac, Bc, r, 0.5, dX, acc, dA, dB, ws)
        assert binding.qlora_workspace_status(ws) == 0
        return dA, dB

    dX = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    dA, dB = run(dX)
    only_a, _ = run(db=False)
    _, only_b = run(da=False)
    assert torch.equal(dB, only_b)
    assert (only_a - dA).norm() <= 4e-6 * dA.norm()  # V comes from another kernel when dB is not asked for
    start = workloads.normal_bf16((M, K), 1.0, 9).cuda()
    acc = start.clone()
    run(acc, 1)
    st = nf4.quantize_weight(W.numpy())
    Wh = nf4.bf16_bits_to_f32(nf4.dequantize_weight(st, "bf16")).astype(np.float64)
    ref, _, _, _ = lora.lora_backward(_f64(x), _f64(dY), Wh, _f64(A), _f64(B), 0.5)
    # The rank step takes s V as bf16 (half a step, 2^-8, of each of its values), the sum of N + r products is fp32
    # (2^-24 each), and the output is rounded once (2^-8).
    v = np.abs(0.5 * _f64(dY) @ _f64(B))
    total = ref + _f64(start)
    inner = 2.0**-8 * v @ np.abs(_f64(A)) + (N + r) * 2.0**-24 * (np.abs(_f64(dY)) @ np.abs(Wh) + v @ np.abs(_f64(A)))
    err = np.abs(_f64(acc) - total)
    assert (err <= inner + 2.0**-8 * (np.abs(total) + inner)).all(), (err - inner - 2.0**-8 * np.abs(total)).max()
    with binding.weight_path(binding.WEIGHT_PATH_DENSE):
        dense = torch.empty_like(dX)
        d1, d2 = run(dense, ws=workspace(M, N, K, r))
    assert torch.equal(dense, dX) and torch.equal(d1, dA) and torch.equal(d2, dB)


def test_nan_stays_in_its_block():
    M, N, K, r = 40, 64, 256, 4
    W, A, B, dY, x = _linear(M, N, K, r, 8)
    x[7, 130] = float("nan")
    w, a, ws = gpu_quantize(W), _checkpoint(x, "int8"), workspace(M, N, K, r)
    dA = torch.empty((r, K), device="cuda")
    binding.qlora_linear_bwd_act8(w, a, dY.cuda(), A.cuda(), B.cuda(), r, 1.0, None, 0, dA, None, ws,
                                  U=torch.zeros((M, r), device="cuda"))
    nan = torch.isnan(dA)
    assert nan[:, 128:192].all() and not nan[:, :128].any() and not nan[:, 192:].any()


@pytest.mark.parametrize("r, with_dx", [(16, False), (40, False), (8, True), (40, True)])
def test_captured_and_on_another_stream(r, with_dx):
    """A captured backward replays to the eager result, on a stream of its own, with new inputs in place."""
    M, N, K = 200, 128, 512
    W, A, B, dY, x = _linear(M, N, K, r, 21)
    w, ws = gpu_quantize(W), workspace(M, N, K, r)
    a = binding.Act8.empty(M, K)
    xc, dYc, Ac, Bc = x.cuda(), dY.cuda(), A.cuda(), B.cuda()
    dA, dB = torch.zeros((r, K), device="cuda"), torch.zeros((N, r), device="cuda")
    dX = torch.empty((M, K), dtype=torch.bfloat16, device="cuda") if with_dx else None

    def step():
        binding.qlora_act8_quantize(xc, a)
        binding.qlora_linear_bwd_act8(w, a, dYc, Ac, Bc, r, 1.0, dX, 0, dA, dB, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in (0, 1):
        xc.copy_((x * (1 + k)).cuda())
        step()
        want = dA.clone(), dB.clone()
        dA.zero_(), dB.zero_()
        graph.replay()
        assert torch.equal(dA, want[0]) and torch.equal(dB, want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(dA, want[0]) and torch.equal(dB, want[1])


@pytest.mark.parametrize("r", [8, 24, 64])
def test_calls_in_a_row_share_a_workspace(r):
    """Two problems in turn on one workspace, nothing waited for in between: each call's kernels overlap, the calls do
    not."""
    M, N, K = 1300, 264, 1088
    problems = []
    for seed in (1, 2):
        W, A, B, dY, x = _linear(M, N, K, r, seed)
        w, a = gpu_quantize(W), _checkpoint(x, list(FORMATS)[seed - 1])
        problems.append((w, a, dY.cuda(), A.cuda(), B.cuda()))
    ws = workspace(M, N, K, r)

    def call(problem):
        w, a, dY, A, B = problem
        out = (torch.empty((M, K), dtype=torch.bfloat16, device="cuda"), torch.empty((r, K), device="cuda"),
               torch.empty((N, r), device="cuda"))
        binding.qlora_linear_bwd_act8(w, a, dY, A, B, r, 1.0, out[0], 0, out[1], out[2], ws)
        return out

    want = []
    for problem in problems:
        want.append(call(problem))
        torch.cuda.synchronize()
    got = [call(problems[i % 2]) for i in range(24)]
    assert binding.qlora_workspace_status(ws) == 0
    for i, out in enumerate(got):
        assert all(torch.equal(p, q) for p, q in zip(out, want[i % 2])), i
