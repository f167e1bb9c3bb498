"""GPU: the operators in the order a fine-tuning step runs them.

    residual norm (+ checkpoint of its output) -> adapted linear head
    -> token log probabilities -> their gradient -> the head's backward from
    the checkpoint -> residual norm backward

once eagerly and once captured, against the same chain in fp64 (with the
checkpoint's values where the backward reads them)."""

import numpy as np
import pytest
import torch

from bit_nf4_quantized_blk_b200 import binding, workloads
from gpu_helpers import gpu_quantize, require_gpu, workspace
from oracle import act8, blocks, lora, nf4

pytestmark = pytest.mark.gpu

M, D, V, N, R, S, EPS = 101, 320, 997, 1000, 8, 2.0, 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _f64(t):
    return t.detach().double().cpu().numpy()


class Chain:
    def __init__(self, fmt):
        g = torch.Generator().manual_seed(3)
        rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.W = workloads.normal_f32((N, D), 0.02, 1)
        self.w = gpu_quantize(self.W)
        self.A = workloads.normal_bf16((R, D), 0.05, 2).cuda()
        self.B = workloads.normal_bf16((N, R), 0.05, 3).cuda()
        self.h, self.y = rand(M, D).to(torch.bfloat16).cuda(), rand(M, D).to(torch.bfloat16).cuda()
        self.w_post, self.gate, self.w_pre = ((1 + 0.1 * rand(D)).cuda() for _ in range(3))
        self.targets = torch.randint(0, V, (M,), generator=g)
        self.targets[::7] = -100
        self.targets = self.targets.cuda()
        scored = (self.targets >= 0).float()
        self.g_logprob = -scored / scored.sum()
        self.g_entropy = torch.full((M,), -0.01 / M, device="cuda")
        e = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        b = torch.bfloat16
        self.h_out, self.x, self.r1, self.r2 = e(M, D, dtype=b), e(M, D, dtype=b), e(M), e(M)
        self.act = binding.Act8.empty(M, D, fmt=fmt)
        self.logits, self.U = e(M, N, dtype=b), e(M, R)
        self.logprob, self.entropy, self.row_max, self.log_sum = e(M), e(M), e(M), e(M)
        self.dlogits = torch.zeros((M, N), dtype=b, device="cuda")  # the padded columns stay zero
        self.dx, self.dA, self.dB = e(M, D, dtype=b), e(R, D), e(N, R)
        self.dh, self.dy = e(M, D, dtype=b), e(M, D, dtype=b)
        self.dw_post, self.dgate, self.dw_pre = e(D), e(D), e(D)
        self.ws = workspace(M, N, D, R)
        self.nws = e(binding.qlora_residual_norm_ws_bytes(M, D), dtype=torch.uint8)

    def run(self):
        q = binding
        q.qlora_residual_norm_fwd(self.h, self.y, self.w_post, self.gate, 0.5, self.w_pre, EPS, self.h_out, self.x,
                                  self.act, self.r1, self.r2)
        q.qlora_linear_fwd(self.w, self.x, self.A, self.B, R, S, self.logits, self.U, self.ws)
        z = self.logits[:, :V]
        q.qlora_token_logprobs_fwd(z, self.targets, 1.0, self.logprob, self.entropy, self.row_max, self.log_sum, 0,
                                   None, None)
        q.qlora_token_logprobs_bwd(z, self.targets, 1.0, self.row_max, self.log_sum, self.entropy, self.g_logprob,
                                   self.g_entropy, self.dlogits[:, :V])
        q.qlora_linear_bwd_act8(self.w, self.act, self.dlogits, self.A, self.B, R, S, self.dx, 0, self.dA, self.dB,
                                self.ws, U=self.U)
        q.qlora_residual_norm_bwd(None, self.dx, self.h_out, self.y, self.w_post, self.gate, 0.5, self.w_pre, self.r1,
                                  self.r2, self.dh, self.dy, self.dw_post, self.dgate, self.dw_pre, self.nws)

    def outputs(self):
        return {k: getattr(self, k) for k in ("x", "logprob", "entropy", "dA", "dB", "dh", "dy", "dw_post", "dgate",
                                             "dw_pre")}


@pytest.mark.parametrize("fmt, name", [(binding.ACT8_INT8, "int8"), (binding.ACT8_E4M3, "e4m3")])
def test_chain(fmt, name):
    c = Chain(fmt)
    c.run()
    assert binding.qlora_workspace_status(c.ws) == 0
    st = nf4.quantize_weight(c.W.numpy())
    Wh = nf4.bf16_bits_to_f32(nf4.dequantize_weight(st, "bf16")).astype(np.float64)
    A, B = _f64(c.A), _f64(c.B)
    norm = (_f64(c.h), _f64(c.y), _f64(c.w_post), _f64(c.gate), 0.5, _f64(c.w_pre))
    v, x, r1, r2 = blocks.residual_norm_forward(*norm, EPS)
    Y, _ = lora.lora_forward(x, Wh, A, B, S)
    t = c.targets.cpu().numpy()
    f = blocks.token_logprobs(Y[:, :V], t, 1.0)
    dY = np.zeros((M, N))
    dY[:, :V] = blocks.token_logprobs_backward(Y[:, :V], t, 1.0, _f64(c.g_logprob), _f64(c.g_entropy))
    dx, _, dB, Vr = lora.lora_backward(x, dY, Wh, A, B, S)
    xh = act8.decode(*act8.encode(act8.round_bf16(x), name), name).reshape(M, D)
    ref = {"x": x, "logprob": f["logprob"], "entropy": f["entropy"], "dA": S * Vr.T @ xh, "dB": dB,
           **blocks.residual_norm_backward(None, dx, v, *norm[1:4], 0.5, norm[5], r1, r2)}
    # bf16 is rounded to at x, the logits (|z| < 4: p off by up to 4 2^-8), dlogits, dx, the rank step and h_out: five
    # values of 2^-8 and one of 2^-6 at most, which do not add up in one direction; their sum bounds the norm.
    for k, got in c.outputs().items():
        err = np.linalg.norm(_f64(got) - ref[k]) / np.linalg.norm(ref[k])
        assert err <= 5 * 2.0**-8 + 2.0**-6, (k, err)
    assert (c.dlogits[:, V:] == 0).all()


def test_captured_chain_with_new_inputs():
    c = Chain(binding.ACT8_INT8)
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    c.y.mul_(-0.5)
    c.targets.copy_(c.targets.flip(0))
    c.run()
    want = {k: v.clone() for k, v in c.outputs().items()}
    for v in c.outputs().values():
        v.zero_()
    graph.replay()
    for k, v in c.outputs().items():
        assert torch.equal(v, want[k]), k


def test_two_chains_at_once():
    """Two chains on two streams, each with its own buffers, give the serial bits."""
    a, b = Chain(binding.ACT8_INT8), Chain(binding.ACT8_E4M3)
    a.run(), b.run()
    want = [{k: v.clone() for k, v in c.outputs().items()} for c in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for c, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                c.run()
    torch.cuda.synchronize()
    for c, w in zip((a, b), want):
        for k, v in c.outputs().items():
            assert torch.equal(v, w[k]), k
