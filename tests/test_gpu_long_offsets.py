"""GPU: element offsets beyond 2^32.  The last rows of a long input get what the
same rows get alone."""

import pytest
import torch

from bit_nf4_quantized_blk_b200 import binding
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
TAIL = 5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def _long(rows, cols, seed):
    """Zeros but for the last TAIL rows."""
    x = torch.zeros((rows, cols), dtype=BF16, device="cuda")
    x[-TAIL:] = torch.randn((TAIL, cols), generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()
    return x


@pytest.mark.parametrize("fmt", [binding.ACT8_INT8, binding.ACT8_E4M3])
def test_checkpoint(fmt):
    D = 8192
    M = (1 << 32) // D + TAIL
    x = _long(M, D, 1)
    ckpt, alone = binding.Act8.empty(M, D, fmt=fmt), binding.Act8.empty(TAIL, D, fmt=fmt)
    binding.qlora_act8_quantize(x, ckpt)
    binding.qlora_act8_quantize(x[-TAIL:], alone)
    assert torch.equal(ckpt.codes[-TAIL:], alone.codes) and torch.equal(ckpt.step[-TAIL:], alone.step)
    assert not ckpt.step[:TAIL].any()
    back = torch.empty((TAIL, D), dtype=BF16, device="cuda")
    binding.qlora_act8_dequantize(alone, back)
    x.fill_(1.0)
    binding.qlora_act8_dequantize(ckpt, x)
    assert torch.equal(x[-TAIL:], back) and not x[:-TAIL].any()


def test_residual_norm():
    D = 8192
    M = (1 << 32) // D + TAIL
    g = torch.Generator().manual_seed(2)
    h, y = _long(M, D, 3), _long(M, D, 4)
    w_post, w_pre, gate = (torch.randn(D, generator=g).cuda() for _ in range(3))

    def forward(h, y, rows):
        x = torch.empty((rows, D), dtype=BF16, device="cuda")
        rstd = [torch.empty(rows, device="cuda") for _ in range(2)]
        binding.qlora_residual_norm_fwd(h, y, w_post, gate, 0.5, w_pre, 1e-5, h, x, None, *rstd)  # in place
        return x, rstd

    few_h = h[-TAIL:].clone()
    few_x, few_rstd = forward(few_h, y[-TAIL:], TAIL)
    x, rstd = forward(h, y, M)
    assert torch.equal(x[-TAIL:], few_x) and torch.equal(h[-TAIL:], few_h)
    assert all(torch.equal(a[-TAIL:], b) for a, b in zip(rstd, few_rstd))

    def backward(dx, h_out, y, rstd, dy):
        dh = torch.zeros_like(h_out)  # the gradient of h_out, in place
        binding.qlora_residual_norm_bwd(dh, dx, h_out, y, w_post, gate, 0.5, w_pre, *rstd, dh, dy, None, None, None, None)
        return dh

    few_dy = torch.empty_like(few_x)
    few_dh = backward(few_x, few_h, y[-TAIL:], few_rstd, few_dy)
    dy = torch.empty_like(x)
    dh = backward(x, h, y, rstd, dy)
    assert torch.equal(dh[-TAIL:], few_dh) and torch.equal(dy[-TAIL:], few_dy)


def test_token_logprobs():
    V = 1 << 17
    M = (1 << 32) // V + TAIL
    x = _long(M, V, 5)
    t = torch.full((M,), V - 1, device="cuda")
    logprob, entropy, m, s = (torch.empty(M, device="cuda") for _ in range(4))
    ids = torch.empty((M, 4), dtype=torch.int32, device="cuda")
    top = torch.empty((M, 4), device="cuda")
    binding.qlora_token_logprobs_fwd(x, t, 1.0, logprob, entropy, m, s, 4, ids, top)
    want = torch.log_softmax(x[-TAIL:].double(), 1)
    order = torch.sort(x[-TAIL:], dim=1, descending=True, stable=True).indices[:, :4]
    assert torch.equal(ids[-TAIL:].long(), order)
    # At most (V / 256 + 32) additions in a chain and the exponentials' 2^-20, all of one sign.
    tol = (V / 256 + 64) * 2.0**-24 + 2.0**-20
    assert (logprob[-TAIL:] - want[:, -1]).abs().max() <= tol + 2.0**-22 * 20
    assert (top[-TAIL:] - want.gather(1, order)).abs().max() <= tol + 2.0**-22 * 20
    g = torch.ones(M, device="cuda")
    binding.qlora_token_logprobs_bwd(x, t, 1.0, m, s, None, g, None, x)  # in place
    grad = -want.exp()
    grad[:, -1] += 1.0
    assert ((x[-TAIL:] - grad).abs() <= (2.0**-8 + 4 * tol) * grad.abs() + 2.0**-24).all()
    assert torch.equal(x[:2, :2], torch.full((2, 2), -1.0 / V, dtype=BF16, device="cuda"))
