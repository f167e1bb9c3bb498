"""GPU: token log probabilities, entropy, alternatives and their gradient
against fp64."""

import numpy as np
import pytest
import torch

from bit_nf4_quantized_blk_b200 import binding
from gpu_helpers import require_gpu
from oracle import blocks

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
DTYPES = [BF16, FP32]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _logits(M, V, dtype, seed, pad=0, std=2.5):
    """[M, V] view of rows padded to a multiple of 8 and `pad` more vectors; the padding holds NaN."""
    g = torch.Generator().manual_seed(seed)
    full = torch.full((M, (V + 7) // 8 * 8 + 8 * pad), float("nan"), dtype=dtype)
    full[:, :V] = (torch.randn((M, V), generator=g) * std).to(dtype)
    return full.cuda()[:, :V]


def _targets(M, V, seed):
    t = torch.randint(0, V, (M,), generator=torch.Generator().manual_seed(seed))
    if M > 3:
        t[::3] = -100
    t[0] = V - 1
    return t.cuda()


def _forward(x, t, it=1.0, k=0):
    M = x.shape[0]
    out = {n: torch.full((M + 1,), 7.0, device="cuda") for n in ("logprob", "entropy", "row_max", "log_sum")}
    ids = torch.full((M * k + 1,), -7, dtype=torch.int32, device="cuda") if k else None
    lps = torch.full((M * k + 1,), 7.0, device="cuda") if k else None
    binding.qlora_token_logprobs_fwd(x, t, it, out["logprob"], out["entropy"], out["row_max"], out["log_sum"], k, ids, lps)
    for v in out.values():
        assert v[M] == 7.0
    out = {n: v[:M] for n, v in out.items()}
    if k:
        assert ids[M * k] == -7 and lps[M * k] == 7.0
        out["top_ids"], out["top_logprob"] = ids[:M * k].view(M, k), lps[:M * k].view(M, k)
    return out


def _same_special(got, ref):
    """Equal where the reference is not finite; returns the finite places."""
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine], ref[~fine], equal_nan=True)
    assert np.isfinite(got[fine]).all()
    return fine


def _sum_error(V):
    """Relative error of sum exp(t): 2^-21 for each exponential, 2^-23 |t| for its argument (terms beyond |t| = 40 are
    below 2^-40 of the sum), and one fp32 addition per term of a thread and step of the joins."""
    return 2.0**-21 + 40 * 2.0**-23 + (V / 256 + 32) * 2.0**-24


def _check_forward(x, t, it=1.0, k=0):
    got = _forward(x, t, it, k)
    ref = blocks.token_logprobs(_f64(x), t.cpu().numpy(), np.float64(np.float32(it)), k)
    V = x.shape[1]
    rel = _sum_error(V)
    if k:
        assert np.array_equal(got["top_ids"].cpu().numpy(), ref["top_ids"])
    assert np.array_equal(_f64(got["row_max"]), ref["row_max"], equal_nan=True)
    for name in ("logprob", "entropy", "log_sum") + (("top_logprob",) if k else ()):
        g, r = _f64(got[name]), ref[name]
        with np.errstate(over="ignore"):
            r = np.where(np.isinf(r.astype(np.float32)), r.astype(np.float32), r)  # beyond fp32: its infinity
        fine = _same_special(g, r)
        # log s: the sum's relative error; the entropy has (sum e t) / s beside it, at most log V + 1 in size; a
        # difference with x: two roundings of its own size.
        size = 3 * (np.log(V) + 1) if name == "entropy" else 1.0
        tol = rel * size + 2.0**-22 * (np.abs(r[fine]) + np.log(V))
        assert (np.abs(g[fine] - r[fine]) <= tol).all(), (name, np.abs(g[fine] - r[fine]).max())
    return got, ref


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M, V, k", [(1, 1, 1), (5, 2, 2), (3, 7, 7), (4, 8, 3), (2, 9, 9), (7, 33, 32), (9, 100, 20),
                                     (3, 513, 5), (2, 1000, 32), (3, 2049, 1), (150, 4100, 20), (3, 8192, 32),
                                     (2, 50257, 20), (1, 131072, 20), (9, 128256, 0)])
def test_forward(M, V, k, dtype):
    _check_forward(_logits(M, V, dtype, M * V, pad=M % 3), _targets(M, V, M + V), k=k)


@pytest.mark.parametrize("it", [0.1, 1.25, 30.0])
def test_temperature(it):
    _check_forward(_logits(6, 3001, FP32, 1), _targets(6, 3001, 2), it, 10)


@pytest.mark.parametrize("it", [2.0**-100, 2.0**100])
@pytest.mark.parametrize("dtype", DTYPES)
def test_extreme_temperature(dtype, it):
    x = _logits(6, 1000, dtype, 31)
    t = _targets(6, 1000, 32)
    x[1, 7] = x[1, 500] = 40.0  # two maxima share the row at low temperature
    _check_forward(x, t, it=it, k=2)


def test_large_and_shifted_logits():
    for shift in (-3e4, 2e5):
        x = _logits(4, 1500, FP32, 3)
        x.add_(shift)
        _check_forward(x, _targets(4, 1500, 4), k=4)


@pytest.mark.parametrize("dtype", DTYPES)
def test_masks(dtype):
    V, k = 2500, 8
    x = _logits(10, V, dtype, 5)
    low = torch.finfo(dtype).min
    x[0, 5:] = float("-inf")  # fewer live logits than alternatives
    x[1, :-1] = float("-inf")  # one live logit, the last
    x[2] = float("-inf")  # none
    x[3] = low  # all at the type's lowest value: an ordinary, uniform row
    x[4, 100:] = low
    x[5, ::2] = low
    x[5, 1::2] = float("-inf")
    x[6, 17:] = float("-inf")
    x[6, 17] = low
    x[7, :1300] = low  # far below the rest
    x[8] = torch.finfo(dtype).max
    x[8, 1::2] = low
    t = torch.tensor([3, V - 1, 0, 7, 2000, 4, 17, 2400, 1, -1], device="cuda")
    got, ref = _check_forward(x, t, k=k)
    assert got["entropy"][2] == 0 and got["logprob"][2] == float("-inf")
    assert abs(got["logprob"][3].item() + np.log(V)) < 1e-5


@pytest.mark.parametrize("dtype", DTYPES)
def test_nonfinite_rows(dtype):
    V = 1700
    x = _logits(8, V, dtype, 6)
    x[0, 900] = float("nan")
    x[1, 3] = float("inf")
    x[2, [5, 1600]] = float("nan")
    x[3, 40:] = float("-inf")
    x[3, 1] = float("nan")
    x[4, 9] = float("inf")
    x[4, 8] = float("nan")
    x[6] = float("nan")
    _check_forward(x, torch.tensor([1, 3, 5, 6, 7, V, 2, V + 5], device="cuda"), k=6)


@pytest.mark.parametrize("dtype", DTYPES)
def test_ties_take_the_lowest_id(dtype):
    for V in (40, 3000, 20000):
        x = torch.zeros((4, (V + 7) // 8 * 8), dtype=dtype)
        x[1, ::2] = -0.0  # equal to 0
        x[2] = torch.arange(x.shape[1]) % 3
        x[3, V // 2:] = 1.0
        x = x.cuda()[:, :V]
        _check_forward(x, _targets(4, V, 1), k=32)


def test_largest_logits_in_one_place():
    """Ascending and descending rows, and all large logits in the vectors of few threads."""
    V = 40000
    x = torch.empty((5, V))
    x[0] = torch.arange(V)
    x[1] = -torch.arange(V)
    x[2] = torch.randn(V, generator=torch.Generator().manual_seed(1))
    x[2].view(-1, 8)[5::256] += 50.0
    x[3] = x[2].flip(0)
    x[4] = 0.0
    x[4].view(-1, 8)[::256] = 1.0
    for dtype in DTYPES:
        _check_forward((x / 64).to(dtype).cuda(), _targets(5, V, 1), k=20)


def _mixed_rows(M, V, dtype, seed):
    """Ordinary rows with masked, tied, empty and NaN ones between them."""
    x, t = _logits(M, V, dtype, seed, pad=1), _targets(M, V, seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    kind = torch.randint(0, 12, (M,), generator=g).cuda()
    x[kind == 0] = 0.5  # ties everywhere: more at the bound than a list holds
    x[kind == 1] = float("-inf")
    x[kind == 2, V // 3] = float("nan")
    half = (kind == 3).nonzero().ravel()
    x[half, : V // 2] = float("-inf")
    x[(kind == 4).nonzero().ravel(), V - 1] = 60.0
    t[kind == 5] = V + 3
    return x, t


@pytest.mark.parametrize("M, V, k, dtype", [(2000, 3001, 0, BF16), (2000, 3001, 5, FP32), (1300, 3001, 32, BF16),
                                            (20000, 40, 5, BF16), (20000, 40, 0, FP32)])
def test_rows_that_follow_each_other(M, V, k, dtype):
    """More rows than CTAs: a CTA's copies run across rows' ends, its counts and lists are used again, and past 32 of
    its rows (20000) its targets are fetched again."""
    _check_forward(*_mixed_rows(M, V, dtype, M + k), k=k)


def test_outputs_left_out():
    x, t = _logits(6, 777, BF16, 9), _targets(6, 777, 1)
    full = _forward(x, t, 0.7, 5)
    M, k = 6, 5
    new = lambda: torch.empty(M, device="cuda")  # noqa: E731
    a, b, c = new(), new(), new()
    binding.qlora_token_logprobs_fwd(x, t, 0.7, a, None, None, None, 0, None, None)
    binding.qlora_token_logprobs_fwd(x, None, 0.7, None, b, None, c, 0, None, None)
    ids, lps = torch.empty((M, k), dtype=torch.int32, device="cuda"), torch.empty((M, k), device="cuda")
    binding.qlora_token_logprobs_fwd(x, None, 0.7, None, None, None, None, k, ids, lps)
    assert torch.equal(a, full["logprob"]) and torch.equal(b, full["entropy"]) and torch.equal(c, full["log_sum"])
    assert torch.equal(ids, full["top_ids"]) and torch.equal(lps, full["top_logprob"])


def _check_backward(x, t, it=1.0, entropy=True, logprob=True, in_place=False):
    M, V = x.shape
    ref_x = _f64(x)
    f = _forward(x, t, it)
    g = torch.Generator().manual_seed(M + V)
    gl = torch.randn(M, generator=g).cuda() if logprob else None
    gh = torch.randn(M, generator=g).cuda() if entropy else None
    full = torch.full((M, (V + 7) // 8 * 8 + 8), 9.0, dtype=x.dtype, device="cuda")
    out = x if in_place else full[:, :V]
    binding.qlora_token_logprobs_bwd(x, t if logprob else None, it, f["row_max"], f["log_sum"],
                                     f["entropy"] if entropy else None, gl, gh, out)
    if not in_place:
        assert (full[:, V:] == 9.0).all()
    it64 = np.float64(np.float32(it))
    tn = t.cpu().numpy() if logprob else np.full(M, -1)
    gl64 = _f64(gl) if logprob else np.zeros(M)
    ref = blocks.token_logprobs_backward(ref_x, tn, it64, gl64, _f64(gh))
    got = _f64(out)
    fine = _same_special(got, ref)
    fwd = blocks.token_logprobs(ref_x, tn, it64)
    with np.errstate(invalid="ignore"):
        lp = (ref_x - fwd["row_max"][:, None]) * it64 - fwd["log_sum"][:, None]
        lp = np.maximum(np.nan_to_num(lp, nan=-1000.0), -1000)  # (an empty row's zeros are exact)
        # p is off by its argument's error: 2^-21 |log p| for the products, the forward's error of log s, 2^-21 for exp;
        # (A - B log p) by a few roundings and by the entropy's error.
        mag = np.exp(lp) * it64 * (np.abs(gl64)[:, None] + (0 if gh is None else np.abs(_f64(gh))[:, None]) *
                                   (np.abs(lp) + fwd["entropy"][:, None] + 3 * (np.log(V) + 1)))
        inner = mag * (4 * _sum_error(V) + 2.0**-20 * (1 + np.abs(lp)))
    inner = inner + 2.0**-22 * it64 * np.abs(gl64)[:, None] + 1e-37
    half = 2.0**-8 if x.dtype == BF16 else 2.0**-24
    err = np.abs(got - ref)[fine] - (inner + half * (np.abs(ref) + inner))[fine]
    assert (err <= 0).all(), err.max()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M, V", [(1, 1), (3, 7), (4, 8), (2, 9), (7, 333), (3, 4097), (40, 8200), (2, 50257)])
@pytest.mark.parametrize("entropy, logprob", [(True, True), (False, True), (True, False)])
def test_backward(M, V, dtype, entropy, logprob):
    _check_backward(_logits(M, V, dtype, M + V), _targets(M, V, V), 0.8, entropy, logprob)


@pytest.mark.parametrize("dtype", DTYPES)
def test_backward_in_place_and_masked(dtype):
    V = 1111
    x = _logits(8, V, dtype, 2)
    low = torch.finfo(dtype).min
    x[0, 5:] = float("-inf")
    x[1] = float("-inf")
    x[2] = low
    x[3, ::2] = low
    x[4, 7] = float("nan")
    x[5, 8] = float("inf")
    t = torch.tensor([2, 3, 4, 5, 6, 7, V, -1], device="cuda")
    _check_backward(x.clone(memory_format=torch.preserve_format) if x.is_contiguous() else x, t, in_place=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("logprob", [True, False])
def test_targets_past_the_end_of_masked_rows(dtype, logprob):
    """A target of V or more gives NaN in every row, an empty one too; a negative one 0 in every row."""
    V = 700
    x = _logits(9, V, dtype, 12)
    x[:4] = float("-inf")
    x[4:7, 5] = float("nan")
    t = torch.tensor([V, -1, 3, V + 100, V, -1, 4, V, -1], device="cuda")
    got, ref = _check_forward(x, t, k=2)
    assert np.isnan(ref["logprob"][[0, 3, 4, 7]]).all() and (ref["logprob"][[1, 5, 8]] == 0).all()
    _check_backward(x, t, logprob=logprob)
    if logprob:
        g = torch.ones(9, device="cuda")
        d = torch.empty((9, 704), dtype=dtype, device="cuda")[:, :V]
        binding.qlora_token_logprobs_bwd(x, t, 1.0, got["row_max"], got["log_sum"], None, g, None, d)
        assert torch.isnan(d[[0, 3, 4, 5, 6, 7]]).all() and (d[[1, 2]] == 0).all() and torch.isfinite(d[8]).all()


def test_gradient_against_differences():
    """The formula itself: central differences of the fp64 forward."""
    rng = np.random.RandomState(0)
    x, t, it = rng.randn(3, 11), np.array([4, -1, 10]), 0.7
    gl, gh = rng.randn(3), rng.randn(3)

    def loss(x):
        f = blocks.token_logprobs(x, t, it)
        return (gl * f["logprob"]).sum() + (gh * f["entropy"]).sum()

    grad = blocks.token_logprobs_backward(x, t, it, gl, gh)
    for i in range(3):
        for j in range(11):
            d = np.zeros_like(x)
            d[i, j] = 1e-5
            assert abs((loss(x + d) - loss(x - d)) / 2e-5 - grad[i, j]) < 1e-8


def test_captured_and_on_another_stream():
    x, t = _logits(20, 5000, BF16, 3), _targets(20, 5000, 1)
    out = [torch.empty(20, device="cuda") for _ in range(4)]
    ids, lps = torch.empty((20, 3), dtype=torch.int32, device="cuda"), torch.empty((20, 3), device="cuda")
    g = torch.ones(20, device="cuda")
    d = torch.empty((20, 5000), dtype=BF16, device="cuda")

    def step():
        binding.qlora_token_logprobs_fwd(x, t, 1.0, *out, 3, ids, lps)
        binding.qlora_token_logprobs_bwd(x, t, 1.0, out[2], out[3], out[1], g, g, d)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.mul_(0.5)
    step()
    want = [v.clone() for v in (*out, ids, lps, d)]
    for v in (*out, ids, lps, d):
        v.zero_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip((*out, ids, lps, d), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip((*out, ids, lps, d), want))
