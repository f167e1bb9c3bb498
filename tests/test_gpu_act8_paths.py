"""GPU: the linear backward from a checkpoint where its products take another path through the workspace and the
pipeline than a few hundred tokens do."""

import pytest
import torch

from bit_nf4_quantized_blk_b200 import binding
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
FORMATS = {"int8": binding.ACT8_INT8, "e4m3": binding.ACT8_E4M3}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()


def _randn(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)


class Problem:
    def __init__(self, M, N, K, r, fmt, seed=0):
        g = torch.Generator(device="cuda").manual_seed(M + N + K + r + seed)
        self.M, self.N, self.K, self.r, self.s = M, N, K, r, 2.0
        self.w = binding.NF4Weight.empty(N, K)
        self.w.packed.random_(0, 256, generator=g)
        self.w.qscale.random_(-127, 128, generator=g)
        self.w.c2.fill_(0.015)
        self.w.mu.fill_(0.045)
        self.A, self.B, self.dY = _randn(g, r, K, std=0.05), _randn(g, N, r, std=0.05), _randn(g, M, N)
        self.a = binding.Act8.empty(M, K, fmt=FORMATS[fmt])
        x = _randn(g, M, K)
        binding.qlora_act8_quantize(x, self.a)
        binding.qlora_act8_dequantize(self.a, x)  # its values
        self.x = x
        self.U = (x.double() @ self.A.double().t()).float()

    def run(self, saved_u, dx=False, da=True, db=True, ws=None):
        M, N, K, r = self.M, self.N, self.K, self.r
        out = [torch.full((M, K), 3.0, dtype=BF16, device="cuda") if dx else None,
               torch.full((r + 1, K), 3.0, device="cuda") if da else None,
               torch.full((N + 1, r), 3.0, device="cuda") if db else None]
        guard = 4096
        if ws is None:
            size = binding.qlora_linear_ws_bytes(M, N, K, r)
            full = torch.full((size + guard,), 0xA5, dtype=torch.uint8, device="cuda")
            ws = full[:size]
            binding.qlora_workspace_reset(ws)
        else:
            full = None
        binding.qlora_linear_bwd_act8(self.w, self.a, self.dY, self.A, self.B, r, self.s, out[0], 0, out[1], out[2], ws,
                                      U=self.U if saved_u else None)
        assert binding.qlora_workspace_status(ws) == 0
        if full is not None:
            assert (full[-guard:] == 0xA5).all()
        for o, rows in ((out[1], r), (out[2], N)):
            if o is not None:
                assert (o[rows] == 3.0).all()
        return out[0], out[1][:r] if da else None, out[2][:N] if db else None

    def check(self, saved_u, da, db):
        """V is an fp32 sum of N products, U (where it is not given) one of K, each output one of 3 M products (three
        bf16 parts, which hold all of V and U): at most (terms) 2^-24 of the sum of magnitudes each."""
        M, N, K = self.M, self.N, self.K
        g, b, a, x = self.dY.double(), self.B.double(), self.A.double(), self.x.double()
        if da is not None:
            ref = self.s * (g @ b).t() @ x
            tol = (N + 3 * M + 2) * 2.0**-24 * self.s * (g.abs() @ b.abs()).t() @ x.abs() + 1e-30
            assert ((da.double() - ref).abs() <= tol).all()
        if db is not None:
            u = self.U.double() if saved_u else x @ a.t()
            absu = u.abs() if saved_u else x.abs() @ a.abs().t()
            ref = self.s * g.t() @ u
            tol = (3 * M + 2 + (0 if saved_u else K)) * 2.0**-24 * self.s * g.abs().t() @ absu + 1e-30
            assert ((db.double() - ref).abs() <= tol).all()


def test_long_inputs_keep_short_chains_of_additions():
    """The tensor core truncates: an addition loses half a unit in the last place of its sum on average, at most 2^-24 of
    it, always in one direction.  dB of 4096 tokens and 131072 outputs adds 48 times in a row (two token tiles, three
    parts), then 8 runs and the token blocks in fp32; all values are positive, so that no sum is larger than its
    result."""
    p = Problem(4096, 131072, 64, 16, "int8")
    for t in (p.dY, p.A, p.B, p.U, p.x):
        t.abs_()
    binding.qlora_act8_quantize(p.x, p.a)
    binding.qlora_act8_dequantize(p.a, p.x)
    for saved_u in (True, False):
        _, _, db = p.run(saved_u, da=False)
        u = p.U.double() if saved_u else p.x.double() @ p.A.double().t()
        ref = torch.zeros_like(db, dtype=torch.float64)
        for i in range(0, p.M, 512):
            ref += p.s * p.dY[i:i + 512].double().t() @ u[i:i + 512]
        terms = 48 + 8 + 2 + (0 if saved_u else 64)
        assert (db.double() - ref).norm() <= terms * 2.0**-24 * ref.norm()


def test_wide_inputs_keep_short_chains_of_additions():
    """V of 65536 outputs at a rank above 16: 64 additions in a row, then 8 sums of those and 8 splits.  X^ has one
    value per column, so that dA is V itself."""
    p = Problem(9600, 65536, 64, 40, "int8")
    p.dY.abs_()
    p.B.abs_()
    p.a.codes.zero_()
    p.a.step.fill_(1.0)
    rows = torch.arange(p.K, device="cuda") * 149
    p.a.codes[rows, torch.arange(p.K, device="cuda")] = 1
    _, da, _ = p.run(True, db=False)
    ref = p.s * (p.dY[rows].double() @ p.B.double()).t()
    assert (da.double() - ref).norm() <= (64 + 8 + 8 + 4) * 2.0**-24 * ref.norm()


@pytest.mark.parametrize("N", [8, 24, 136, 264, 1032])
@pytest.mark.parametrize("r", [33, 48, 64])
def test_columns_that_end_inside_a_warp(N, r):
    """Ranks above 32 take a warp of the column sums' epilogue twice through its loop, and the columns of dB may end
    within the warp: its lanes load the second accumulators together all the same."""
    p = Problem(300, N, 192, r, "int8")
    for saved_u in (True, False):
        _, da, db = p.run(saved_u)
        p.check(saved_u, da, db)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M, N, K, r", [
    (1, 64, 64, 64), (2, 128, 64, 64), (16, 40, 64, 64),  # single splits: no partials of dA
    (40000, 8, 64, 40),                                   # no room for U's and V's partials side by side
    (8000, 128, 14336, 40),                               # room for dB's and dA's with fewer splits
    (8000, 8, 14336, 64),                                 # none side by side, for dA's alone with fewer splits
    (40000, 8, 14336, 8),                                 # the same, ranks up to 16
    (33, 72, 192, 8), (300, 72, 576, 33)])
def test_everything_fits_the_linear_workspace(M, N, K, r, fmt):
    p = Problem(M, N, K, r, fmt)
    for saved_u in (True, False):
        _, da, db = p.run(saved_u)
        p.check(saved_u, da, db)
        _, only_a, _ = p.run(saved_u, db=False)
        p.check(saved_u, only_a, None)
    if M < 1000:  # with the dX GEMM between the products
        dx, da2, db2 = p.run(True, dx=True)
        p.check(True, da2, db2)
        want = torch.empty_like(dx)
        ws = torch.empty(binding.qlora_linear_ws_bytes(M, N, K, r), dtype=torch.uint8, device="cuda")
        binding.qlora_workspace_reset(ws)
        binding.qlora_linear_bwd(p.w, p.x, p.dY, p.A, p.B, r, p.s, want, 0, None, None, ws)
        # Both V are within e = N 2^-24 sum |dY| |B| of the exact one, so their bf16 roundings (2^-8 each) differ by at
        # most 2^-7 (|V| + e) + 2 e; and dX is rounded once on each side.
        e = N * 2.0**-24 * p.dY.double().abs() @ p.B.double().abs()
        v = (p.dY.double() @ p.B.double()).abs()
        apart = p.s * (2.0**-7 * (v + e) + 2 * e) @ p.A.double().abs()
        assert ((dx.double() - want.double()).abs() <= apart + 2.0**-7 * want.double().abs() + 1e-30).all()


# Steps of a CTA (64 tokens each for dA and dB, 128 columns for U and V), of which three are in flight.
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M, N, K, r", [
    (1999, 2048, 8192, 64),  # U 8, V 16, dB 16, dA 8 steps
    (1987, 2056, 8128, 40),  # the same with ragged ends everywhere; V 17
    (1987, 2056, 8128, 11),  # dA 7 or 8; V and dB from one pass
    (6300, 136, 8192, 24),   # dA in two waves of CTAs, 11 steps each
])
def test_products_of_many_steps(M, N, K, r, fmt):
    """Every stage of a product's pipeline is used several times over, the last ones not all equally often."""
    p = Problem(M, N, K, r, fmt)
    ws = torch.empty(binding.qlora_linear_ws_bytes(M, N, K, r), dtype=torch.uint8, device="cuda")
    binding.qlora_workspace_reset(ws)
    first = {}
    for saved_u in (True, False):
        _, da, db = first[saved_u] = p.run(saved_u, ws=ws)
        p.check(saved_u, da, db)
        _, da, _ = p.run(saved_u, db=False, ws=ws)
        p.check(saved_u, da, None)
    for i in range(8):  # in a row on one workspace
        _, da, db = p.run(i % 2 == 0, ws=ws)
        assert torch.equal(da, first[i % 2 == 0][1]) and torch.equal(db, first[i % 2 == 0][2])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M, r", [(2, 3), (16, 8), (16, 64), (32, 8), (32, 40), (66, 16), (200, 64), (1000, 12)])
def test_third_parts_of_u_and_v(M, r, fmt):
    """V and U of token 2 i are those of token 2 i + 1 and 2^-19 more, which their first two bf16 parts do not hold, and
    the other factor is that of token 2 i + 1 negated: what is left of dA and dB is the third parts' product alone.

    Each token's V is base + b1 + 2^-19 with base a bf16 in [1, 2) and b1 one in [2^-10, 2^-9): 2^-19 is below half of
    b1's last place, 2^-17.  The first parts' products cancel exactly, 16 tokens at a time; added to the sum they can
    cost it 2^-22 (one unit of a sum that passes 2 to 4) for each of the 17 terms (the tokens' and the sum).
    """
    N, K = 8, 64
    g = torch.Generator().manual_seed(M + r)
    base = 1 + torch.randint(0, 128, (r,), generator=g) / 128
    b1 = (1 + torch.randint(0, 128, (r,), generator=g) / 128) * 2.0**-10
    even = (torch.arange(M) % 2 == 0).double()
    sign = 2 * even - 1
    tol = (M + 15) // 16 * (min(M, 16) + 1) * 2.0**-22
    one = {"int8": 1, "e4m3": 0x38}[fmt]  # the code of 1
    w = binding.NF4Weight.empty(N, K)
    for t in (w.packed, w.qscale, w.c2, w.mu):
        t.zero_()

    def run(x_codes, dY, A, B, U):
        a = binding.Act8(M, K, x_codes.to(torch.uint8).cuda(), torch.ones((M, K // 64), dtype=BF16, device="cuda"),
                         FORMATS[fmt])
        ws = torch.empty(binding.qlora_linear_ws_bytes(M, N, K, r), dtype=torch.uint8, device="cuda")
        binding.qlora_workspace_reset(ws)
        dA, dB = torch.empty((r, K), device="cuda"), torch.empty((N, r), device="cuda")
        f = lambda t: t.to(BF16).cuda().contiguous()  # noqa: E731
        binding.qlora_linear_bwd_act8(w, a, f(dY), f(A), f(B), r, 1.0, None, 0, dA, dB, ws,
                                      U=None if U is None else U.float().cuda())
        assert binding.qlora_workspace_status(ws) == 0
        return dA.double().cpu(), dB.double().cpu()

    # dA: V from dY and B; X^ in +-[1, 2): int8 codes of +-1, E4M3 codes of 1 + i / 8
    if fmt == "int8":
        x = torch.ones((M, K), dtype=torch.float64)
        codes = torch.where(even[:, None] > 0, 1, 255).expand(M, K)
    else:
        eighths = torch.randint(0, 8, (1 + M // 2, K), generator=g).repeat_interleave(2, 0)[:M]
        x = 1 + eighths.double() / 8
        codes = torch.where(even[:, None] > 0, 0x38 + eighths, 0xB8 + eighths)
    dY = torch.zeros((M, N))
    dY[:, :2], dY[:, 2] = 1.0, even
    B = torch.zeros((N, r))
    B[0], B[1], B[2] = base, b1, 2.0**-19
    want = (2.0**-19 * even[:, None] * x).sum(0).expand(r, K)
    assert (want > 2 * tol).all()  # a result without the third parts, zero, would not pass
    dA, _ = run(codes, dY, torch.zeros((r, K)), B, torch.zeros((M, r)))
    assert ((dA - want).abs() <= tol).all()

    # dB: U saved, or from X^ and A; dY in +-[1, 2)
    y = 1 + torch.randint(0, 128, (1 + M // 2, N), generator=g).repeat_interleave(2, 0)[:M].double() / 128
    want = (2.0**-19 * even[:, None] * y).sum(0)[:, None].expand(N, r)
    assert (want > 2 * tol).all()
    codes = torch.zeros((M, K), dtype=torch.int64)
    codes[:, :2], codes[:, 2] = one, (one * even).long()
    A = torch.zeros((r, K))
    A[:, 0], A[:, 1], A[:, 2] = base, b1, 2.0**-19
    U = base.double() + b1.double() + 2.0**-19 * even[:, None]
    for u in (U, None):
        _, dB = run(codes, sign[:, None] * y, A, torch.zeros((N, r)), u)
        assert ((dB - want).abs() <= tol).all()


@pytest.mark.parametrize("M, N, K, r", [(16, 40, 64, 64), (1, 136, 192, 64), (2100, 264, 1088, 16),
                                        (1987, 2056, 512, 40), (8000, 8, 14336, 64)])
@pytest.mark.parametrize("dx", [False, True])
def test_captured_and_two_at_once(M, N, K, r, dx):
    """A captured backward replays to the eager result, and two on streams of their own, each with its workspace, do
    not meet."""
    p, other = Problem(M, N, K, r, "int8"), Problem(M, N, K, r, "e4m3", seed=1)
    size = binding.qlora_linear_ws_bytes(M, N, K, r)

    def buffers():
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        binding.qlora_workspace_reset(ws)
        return ws, (torch.empty((M, K), dtype=BF16, device="cuda") if dx else None, torch.empty((r, K), device="cuda"),
                    torch.empty((N, r), device="cuda"))

    def call(q, ws, out, stream=None):
        binding.qlora_linear_bwd_act8(q.w, q.a, q.dY, q.A, q.B, r, q.s, out[0], 0, out[1], out[2], ws, stream=stream)

    def same(a, b):
        return all(x is None or torch.equal(x, y) for x, y in zip(a, b))

    want = []
    for q in (p, other):
        ws, out = buffers()
        call(q, ws, out)
        want.append(out)
    torch.cuda.synchronize()
    ws, out = buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(p, ws, out)
        call(p, ws, out)  # on the same workspace
    for _ in range(3):
        for t in out:
            if t is not None:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, want[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    pairs = [buffers() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for q, s, (ws, out) in zip((p, other), streams, pairs):
            call(q, ws, out, stream=s)
    torch.cuda.synchronize()
    for (ws, out), w in zip(pairs, want):
        assert binding.qlora_workspace_status(ws) == 0 and same(out, w)
