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
    (1, 64, 64, 64), (2, 128, 64, 64), (16, 40, 64, 64),  # dB's and dA's partials have no room side by side
    (40000, 8, 64, 40),                                     # nor U's and V's
    (8000, 128, 14336, 40),                                 # room with fewer splits
    (8000, 8, 14336, 64),                                   # dA's alone with fewer splits
    (40000, 8, 14336, 8),                                   # the same, ranks up to 16
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
