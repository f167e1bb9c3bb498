"""GPU: the residual sum between two norms, forward and backward, against fp64."""

import itertools

import numpy as np
import pytest
import torch

from bit_nf4_quantized_blk_b200 import binding
from gpu_helpers import require_gpu
from oracle import act8, blocks

pytestmark = pytest.mark.gpu

EPS = 1e-5
# bf16 and fp32: half a step of the output's rounding.
HALF = {torch.bfloat16: 2.0**-8, torch.float32: 2.0**-24}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


class Case:
    def __init__(self, M, D, res=torch.bfloat16, post=True, gate=True, seed=0, scale=0.75):
        g = torch.Generator().manual_seed(1000 * M + D + seed)

        def rand(*s, std=1.0, mean=0.0):
            return mean + std * torch.randn(s, generator=g)

        self.M, self.D, self.res, self.scale = M, D, res, scale
        self.h = rand(M, D, std=2.0).to(res).cuda()
        self.y = rand(M, D, std=0.5).to(torch.bfloat16).cuda()
        if M > 2:
            self.h[1] = 0.0  # a padded row
            self.y[1] = 0.0
        self.w_post = rand(D, std=0.2, mean=1.0).cuda() if post else None
        self.gate = rand(D, std=0.3, mean=0.2).cuda() if gate else None
        self.w_pre = rand(D, std=0.2, mean=1.0).cuda()
        self.dh_out = rand(M, D, std=0.1).to(res).cuda()
        self.dx = rand(M, D, std=0.1).to(torch.bfloat16).cuda()

    def forward(self, h_out=None, fmt=None, w_pre=True, y=True):
        M, D = self.M, self.D
        self.h_out = torch.empty_like(self.h) if h_out is None else h_out
        self.x = torch.empty((M, D), dtype=torch.bfloat16, device="cuda") if w_pre else None
        self.rstd_post = torch.empty(M, device="cuda") if self.w_post is not None and y else None
        self.rstd_pre = torch.empty(M, device="cuda") if w_pre else None
        self.act = binding.Act8.empty(M, D, fmt=fmt) if fmt is not None else None
        binding.qlora_residual_norm_fwd(self.h, self.y if y else None, self.w_post if y else None,
                                        self.gate if y else None, self.scale, self.w_pre if w_pre else None, EPS,
                                        self.h_out, self.x, self.act, self.rstd_post, self.rstd_pre)
        return self

    def backward(self, want=("dh", "dy", "dw_post", "dgate", "dw_pre"), dh_out=True, dx=True, in_place=False):
        M, D = self.M, self.D
        out = {"dh": torch.empty_like(self.h), "dy": torch.empty_like(self.y)}
        for k in ("dw_post", "dgate", "dw_pre"):
            out[k] = torch.empty(D, device="cuda")
        if self.w_post is None:
            out.pop("dw_post")
        if self.gate is None:
            out.pop("dgate")
        if not dx:
            out.pop("dw_pre")
        out = {k: v for k, v in out.items() if k in want}
        if in_place:
            out["dh"] = self.dh_out
        ws = torch.full((binding.qlora_residual_norm_ws_bytes(M, D),), 0x5A, dtype=torch.uint8, device="cuda")
        binding.qlora_residual_norm_bwd(self.dh_out if dh_out else None, self.dx if dx else None, self.h_out, self.y,
                                        self.w_post, self.gate, self.scale, self.w_pre if dx else None,
                                        self.rstd_post, self.rstd_pre if dx else None, out.get("dh"), out.get("dy"),
                                        out.get("dw_post"), out.get("dgate"), out.get("dw_pre"), ws)
        assert (ws[:256] == 0x5A).all()  # a linear workspace's status word would survive
        return out


def _near(got, ref, half, inner):
    """|got - ref| within one rounding of the output (`half` of the value) after `inner` of absolute error."""
    err = np.abs(_f64(got) - ref)
    tol = inner + half * (np.abs(ref) + inner)
    assert (err <= tol).all(), float((err - tol).max())


# A row sum of D products in fp32, by threads and then by a tree, is off by less than (D / TPR + 16) 2^-24 of its
# magnitudes; 64 units cover every row length here (at most 32 terms per thread), for a sum of squares as for a dot product.
ROW = 64 * 2.0**-24


def _check_forward(c):
    v, x, rstd_post, rstd_pre = blocks.residual_norm_forward(_f64(c.h), _f64(c.y), _f64(c.w_post), _f64(c.gate),
                                                             c.scale, _f64(c.w_pre), EPS)
    branch = np.abs(v - _f64(c.h))
    inner = ROW * (branch + np.abs(v))  # the branch's rstd and products; the sum
    _near(c.h_out, v, HALF[c.res], inner)
    if rstd_post is not None:
        assert (np.abs(_f64(c.rstd_post) - rstd_post) <= ROW * rstd_post).all()
    # v is off by `inner`, its norm by that much of the row, rstd by half of both relative errors
    rel = ROW + np.sqrt((inner**2).mean(1)) * rstd_pre
    assert (np.abs(_f64(c.rstd_pre) - rstd_pre) <= rel * rstd_pre).all()
    _near(c.x, x, HALF[torch.bfloat16], rel[:, None] * np.abs(x) + inner * rstd_pre[:, None] * np.abs(_f64(c.w_pre)))


SHAPES = [(1, 64), (3, 64), (9, 192), (2, 320), (37, 512), (5, 960), (1, 1088), (300, 2048), (3, 2112), (130, 4096),
          (7, 5120), (2, 8192), (3, 10240), (2, 16384)]


@pytest.mark.parametrize("M, D", SHAPES)
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_forward(M, D, res):
    _check_forward(Case(M, D, res).forward())


@pytest.mark.parametrize("post, gate", list(itertools.product([True, False], repeat=2)))
def test_forward_parts(post, gate):
    _check_forward(Case(11, 576, post=post, gate=gate).forward())


def test_forward_without_block_or_next_norm():
    c = Case(6, 448, torch.float32).forward(y=False)  # the first norm of a network
    assert torch.equal(c.h_out, c.h)
    _, x, _, rstd = blocks.residual_norm_forward(_f64(c.h), None, None, None, 1.0, _f64(c.w_pre), EPS)
    _near(c.x, x, HALF[torch.bfloat16], 2 * ROW * np.abs(x))
    assert (np.abs(_f64(c.rstd_pre) - rstd) <= ROW * rstd).all()
    full = Case(6, 448, torch.float32).forward()
    last = Case(6, 448, torch.float32).forward(w_pre=False)  # a residual sum alone
    assert torch.equal(full.h_out, last.h_out)


def test_forward_in_place():
    a, b = Case(50, 1024).forward(), Case(50, 1024)
    b.forward(h_out=b.h)
    assert torch.equal(a.h_out, b.h_out) and torch.equal(a.x, b.x)


@pytest.mark.parametrize("fmt, name", [(binding.ACT8_INT8, "int8"), (binding.ACT8_E4M3, "e4m3")])
@pytest.mark.parametrize("M, D", [(1, 64), (9, 192), (5, 960), (20, 2112), (3, 4096), (2, 16384)])
def test_forward_checkpoint(M, D, fmt, name):
    """The checkpoint is that of x as stored, bit for bit."""
    c = Case(M, D).forward(fmt=fmt)
    codes, step = act8.encode(_f64(c.x), name)
    assert np.array_equal(c.act.codes.cpu().numpy().ravel(), codes)
    assert np.array_equal(_f64(c.act.step).ravel(), step)


def _check_backward(c, got, **kw):
    dh_out = _f64(c.dh_out0) if kw.get("dh_out", True) else None
    dx = _f64(c.dx) if kw.get("dx", True) else None
    args = (dh_out, dx, _f64(c.h_out), _f64(c.y), _f64(c.w_post), _f64(c.gate), c.scale, _f64(c.w_pre),
            _f64(c.rstd_post), _f64(c.rstd_pre))
    ref = blocks.residual_norm_backward(*args)
    # Magnitudes: every product of the formula with its absolute value, which bounds what fp32 loses of it.
    a = [None if v is None or i == 6 else np.abs(v) for i, v in enumerate(args)]
    a[6] = abs(c.scale)
    dn = 0.0 if dx is None else a[1] * a[7]
    n = 0.0 if dx is None else a[2] * a[9][:, None]
    g = (0.0 if dh_out is None else a[0]) + (0.0 if dx is None else
                                            a[9][:, None] * (dn + n * (dn * n).mean(1, keepdims=True)))
    rows = (c.M + 16) * 2.0**-24  # a column sum of M fp32 terms
    if "dh" in got:
        _near(got["dh"], ref["dh"], HALF[c.res], 2 * ROW * g)
    if "dw_pre" in got:
        _near(got["dw_pre"], ref["dw_pre"], 2.0**-24, (ROW + rows) * (a[1] * n).sum(0))
    dp = a[6] * g * (1.0 if a[5] is None else a[5])
    m = a[3] if a[8] is None else a[3] * a[8][:, None]
    if "dgate" in got:
        _near(got["dgate"], ref["dgate"], 2.0**-24,
              (4 * ROW + rows) * (a[6] * g * m * (1.0 if a[4] is None else a[4])).sum(0))
    if "dw_post" in got:
        _near(got["dw_post"], ref["dw_post"], 2.0**-24, (4 * ROW + rows) * (dp * m).sum(0))
    if "dy" in got:
        t = dp if a[4] is None else a[8][:, None] * (dp * a[4] + m * (dp * a[4] * m).mean(1, keepdims=True))
        _near(got["dy"], ref["dy"], 2.0**-8, 6 * ROW * t)


def _forward_backward(c, **kw):
    c.forward()
    c.dh_out0 = c.dh_out.clone()
    got = c.backward(**kw)
    _check_backward(c, got, **{k: v for k, v in kw.items() if k in ("dh_out", "dx")})
    return got


@pytest.mark.parametrize("M, D", SHAPES + [(1500, 256), (700, 1024)])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_backward(M, D, res):
    _forward_backward(Case(M, D, res))


@pytest.mark.parametrize("M, D, res", [(76001, 64, torch.bfloat16), (38001, 576, torch.bfloat16),
                                       (5001, 4096, torch.float32)])
def test_backward_of_many_rows(M, D, res):
    """More than 32 rows for a CTA (or a warp), so that it fetches their scalars a second time, with every column sum."""
    _forward_backward(Case(M, D, res))


@pytest.mark.parametrize("post, gate", list(itertools.product([True, False], repeat=2)))
def test_backward_parts(post, gate):
    _forward_backward(Case(11, 576, post=post, gate=gate))
    _forward_backward(Case(400, 2048, post=post, gate=gate))


@pytest.mark.parametrize("want", [("dh",), ("dy",), ("dw_post",), ("dgate",), ("dw_pre",), ("dh", "dy")])
def test_backward_outputs_left_out(want):
    for D in (576, 2112):
        got = _forward_backward(Case(301, D), want=want)
        assert set(got) == set(want)


def test_backward_upstream_left_out():
    for D in (576, 4096):
        _forward_backward(Case(302, D), dh_out=False)
        _forward_backward(Case(302, D), dx=False)


def test_backward_in_place_and_repeatable():
    a = _forward_backward(Case(600, 2048))
    b = _forward_backward(Case(600, 2048), in_place=True)
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_gradients_against_differences():
    """The formulas themselves: central differences of the fp64 forward."""
    rng = np.random.RandomState(4)
    M, D, scale = 3, 64, 0.6
    h, y = rng.randn(M, D), rng.randn(M, D)
    w_post, gate, w_pre = rng.rand(D) + 0.5, rng.randn(D), rng.rand(D) + 0.5
    dh_out, dx = rng.randn(M, D), rng.randn(M, D)

    def loss(h, y, w_post, gate, w_pre):
        v, x, _, _ = blocks.residual_norm_forward(h, y, w_post, gate, scale, w_pre, EPS)
        return (v * dh_out).sum() + (x * dx).sum()

    v, _, r1, r2 = blocks.residual_norm_forward(h, y, w_post, gate, scale, w_pre, EPS)
    g = blocks.residual_norm_backward(dh_out, dx, v, y, w_post, gate, scale, w_pre, r1, r2)
    args = [h, y, w_post, gate, w_pre]
    for i, name in enumerate(("dh", "dy", "dw_post", "dgate", "dw_pre")):
        for _ in range(5):
            at = tuple(rng.randint(s) for s in args[i].shape)
            d = 1e-5
            moved = [a.copy() for a in args]
            moved[i][at] += d
            up = loss(*moved)
            moved[i][at] -= 2 * d
            assert abs((up - loss(*moved)) / (2 * d) - g[name][at]) < 1e-6 * max(1.0, abs(g[name][at]))


def test_nonfinite_rows_stay_alone():
    c = Case(40, 1088)
    c.y[5, 7] = float("nan")
    c.h[9, 3] = float("inf")
    c.forward()
    bad = ~torch.isfinite(c.x).all(1)
    assert bad.nonzero().ravel().tolist() == [5, 9]


def test_captured_pass():
    c = Case(64, 2048)
    c.forward(fmt=binding.ACT8_INT8)
    ws = torch.empty(binding.qlora_residual_norm_ws_bytes(64, 2048), dtype=torch.uint8, device="cuda")
    dh, dy, dw = torch.empty_like(c.h), torch.empty_like(c.y), [torch.empty(2048, device="cuda") for _ in range(3)]

    def step():
        binding.qlora_residual_norm_fwd(c.h, c.y, c.w_post, c.gate, c.scale, c.w_pre, EPS, c.h_out, c.x, c.act,
                                        c.rstd_post, c.rstd_pre)
        binding.qlora_residual_norm_bwd(c.dh_out, c.dx, c.h_out, c.y, c.w_post, c.gate, c.scale, c.w_pre, c.rstd_post,
                                        c.rstd_pre, dh, dy, *dw, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in (1.0, -0.5):
        c.h.mul_(k)
        step()
        want = [t.clone() for t in (c.x, c.act.codes, dh, dy, *dw)]
        for t in (c.x, c.act.codes, dh, dy, *dw):
            t.zero_()
        graph.replay()
        for t, w in zip((c.x, c.act.codes, dh, dy, *dw), want):
            assert torch.equal(t, w)
