"""The operators around the adapted linear layers, as cases to time and compare.

A fine-tuning step of adapted 4-bit projections runs three things besides the
projections themselves, and each is a family of cases here:

  ckpt   8-bit activation checkpoints: X [M, K] kept as one byte per value and
         one bf16 step per 64 values of a row.
             int8:  step = bf16(absmax / 127),  q = round(x / step),  x^ = bf16(q step)
             e4m3:  step = bf16(absmax / 256),  q = E4M3(x / step),   x^ = bf16(q step)
         (round: ties to even; a block of zeros has step 0 and x^ = 0).
  linear the backward of Y = X W^T + s (X A^T) B^T from such a checkpoint:
             V = dY B,  dX = dY W + s V A,  dA = s V^T X^,  dB = s dY^T U
         with U = X A^T as the forward saved it, or X^ A^T recomputed.
  norm   the norm after a block, its gate and residual scale, the residual sum
         and the norm before the next block:
             p = y rstd(y) w_post,  h' = h + scale gate p,  x = h' rstd(h') w_pre
         with rstd(v) = 1 / sqrt(mean(v^2) + eps), x optionally checkpointed
         too, and the backward pass.
  logp   log probabilities of given tokens, z = logits / temperature:
             logp_t = z_t - lse,  H = lse - sum p z,  the k largest z - lse
         and their gradient  dlogits_j = (g (1[j = t] - p_j)
                                          - g_H p_j (log p_j + H)) / temperature.

``run`` computes a case in plain torch, or, where ``own`` is true, through the
library's entry points.
"""

import math

import torch

own = False

DEVICE = "cuda"
BLOCK = 64
NF4 = (-1.0, -0.6961928009986877, -0.5250730514526367, -0.39491748809814453, -0.28444138169288635,
       -0.18477343022823334, -0.09105003625154495, 0.0, 0.07958029955625534, 0.16093020141124725,
       0.24611230194568634, 0.33791524171829224, 0.44070982933044434, 0.5626170039176941, 0.7229568362236023, 1.0)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One short prompt's input of a 2048-wide layer: launch latency.
        {"name": "ckpt 17x2048 e4m3", "op": "ckpt", "M": 17, "K": 2048, "fmt": "e4m3"},
        # The widest activation of a 7B layer (the down projection's input) at 8192 tokens.
        {"name": "ckpt 8192x14336 int8", "op": "ckpt", "M": 8192, "K": 14336, "fmt": "int8"},
        # The k / v projection of a 7B layer on a few tokens, adapter gradients of a short batch.
        {"name": "linear 33x1024x4096 r8", "op": "linear", "M": 33, "N": 1024, "K": 4096, "r": 8, "fmt": "e4m3",
         "saved_u": True, "dx": True},
        # fc2 of a 2048-wide layer, an odd token count, a wide adapter, U recomputed; the first
        # layer of a network: no gradient of its input.
        {"name": "linear 1999x2048x8192 r64", "op": "linear", "M": 1999, "N": 2048, "K": 8192, "r": 64,
         "fmt": "int8", "saved_u": False, "dx": False},
        # The gate projection of a 7B layer at a training step's 8192 tokens.
        {"name": "linear 8192x14336x4096 r16", "op": "linear", "M": 8192, "N": 14336, "K": 4096, "r": 16,
         "fmt": "int8", "saved_u": True, "dx": True},
        # One token of a 7B layer being served.
        {"name": "norm fwd 1x4096", "op": "norm_fwd", "M": 1, "D": 4096, "res": "bf16", "post": True, "gate": False,
         "ckpt": False},
        # A 7B layer at a training step's tokens, its norm output checkpointed.
        {"name": "norm fwd 8192x4096 ckpt", "op": "norm_fwd", "M": 8192, "D": 4096, "res": "bf16", "post": True,
         "gate": True, "ckpt": True},
        # A ragged batch of a 2048-wide model with an fp32 residual stream and no norm after the block.
        {"name": "norm bwd 999x2048 fp32", "op": "norm_bwd", "M": 999, "D": 2048, "res": "fp32", "post": False,
         "gate": True, "ckpt": False},
        # A 7B layer's training step, every gradient.
        {"name": "norm bwd 8192x4096", "op": "norm_bwd", "M": 8192, "D": 4096, "res": "bf16", "post": True,
         "gate": True, "ckpt": False},
        # One served token with its 20 alternatives, a large vocabulary.
        {"name": "logp fwd 1x131072 top20", "op": "logp_fwd", "M": 1, "V": 131072, "ld": 131072, "dtype": "bf16",
         "top": 20, "temp": 0.8},
        # Scoring a batch: an odd vocabulary in rows padded to the head's multiple of 8.
        {"name": "logp fwd 4096x50257", "op": "logp_fwd", "M": 4096, "V": 50257, "ld": 50264, "dtype": "bf16",
         "top": 5, "temp": 1.0},
        # The loss gradient of a training batch with an entropy term.
        {"name": "logp bwd 2048x131072", "op": "logp_bwd", "M": 2048, "V": 131072, "ld": 131072, "dtype": "bf16",
         "top": 0, "temp": 1.0},
    ]


def _spread(rng, lo, hi, step=1):
    """A whole number spread over the logarithm of [lo, hi], a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(v / step + 0.5) * step))


def draw(rng):
    op = rng.choice(["ckpt", "linear", "norm_fwd", "norm_bwd", "logp_fwd", "logp_bwd"])
    if op == "ckpt":
        return {"op": op, "M": _spread(rng, 1, 8192), "K": _spread(rng, 64, 14336, 64),
                "fmt": rng.choice(["int8", "e4m3"])}
    if op == "linear":
        return {"op": op, "M": _spread(rng, 1, 8192), "N": _spread(rng, 64, 8192, 8),
                "K": _spread(rng, 64, 8192, 64), "r": _spread(rng, 1, 64), "fmt": rng.choice(["int8", "e4m3"]),
                "saved_u": rng.random() < 0.6, "dx": rng.random() < 0.6}
    if op in ("norm_fwd", "norm_bwd"):
        return {"op": op, "M": _spread(rng, 1, 8192), "D": _spread(rng, 64, 8192, 64),
                "res": rng.choice(["bf16", "fp32"]), "post": rng.random() < 0.7, "gate": rng.random() < 0.6,
                "ckpt": op == "norm_fwd" and rng.random() < 0.5}
    V = _spread(rng, 17, 131072)
    fp32 = rng.random() < 0.3
    top = 1 << 27  # values of the largest case
    return {"op": op, "M": max(1, min(_spread(rng, 1, 8192), (top // 2 if fp32 else top) // V)), "V": V,
            "ld": (V + 7) // 8 * 8 + 8 * rng.randrange(3), "dtype": "fp32" if fp32 else "bf16",
            "top": rng.choice([0, 1, 5, 20, 32]) if op == "logp_fwd" and V >= 32 else 0,
            "temp": rng.choice([0.6, 0.8, 1.0, 1.3])}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFF)
    return g


def _randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEVICE) * std).to(dtype)


def _activations(g, M, K):
    """bf16 N(0, 1) with a few large channels and, past a handful of rows, one padded (zero) row."""
    x = torch.randn((M, K), generator=g, device=DEVICE)
    x[:, torch.randint(0, K, (max(1, K // 512),), generator=g, device=DEVICE)] *= 20.0
    if M > 4:
        x[M // 2] = 0.0
    return x.to(torch.bfloat16)


def _checkpoint(x, fmt):
    """(stored codes, steps): the definition at the top of this file."""
    v = x.float().view(x.shape[0], -1, BLOCK)
    step = (v.abs().amax(2) / (127.0 if fmt == "int8" else 256.0)).to(torch.bfloat16)
    d = step.float().unsqueeze(2)
    q = v / torch.where(d > 0, d, torch.ones_like(d))
    q = torch.round(q).to(torch.int8) if fmt == "int8" else q.to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(x.shape), step


def _checkpoint_values(codes, step, fmt):
    """The bf16 values that a checkpoint stands for, in 32 bits."""
    q = codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float().view(codes.shape[0], -1, BLOCK)
    return (q * step.float().unsqueeze(2)).to(torch.bfloat16).float().view(codes.shape)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": dict(case)}
    if op == "ckpt":
        s["x"] = _activations(g, case["M"], case["K"])
    elif op == "linear":
        M, N, K, r = (case[k] for k in ("M", "N", "K", "r"))
        blocks = N * K // BLOCK
        s["packed"] = torch.randint(0, 256, (N * K // 2,), generator=g, device=DEVICE, dtype=torch.uint8)
        s["qscale"] = torch.randint(-127, 128, (blocks,), generator=g, device=DEVICE, dtype=torch.int8)
        s["c2"] = 0.01 + 0.01 * torch.rand((blocks + 255) // 256, generator=g, device=DEVICE)
        s["mu"] = torch.full((1,), 0.045, device=DEVICE)
        s["A"], s["B"] = _randn(g, r, K, std=0.02), _randn(g, N, r, std=0.02)
        x = _activations(g, M, K)
        s["dy"] = _randn(g, M, N)
        s["codes"], s["step"] = _checkpoint(x, case["fmt"])
        s["u"] = x.float() @ s["A"].float().t() if case["saved_u"] else None
        s["scale"] = 32.0 / r
    elif op in ("norm_fwd", "norm_bwd"):
        M, D = case["M"], case["D"]
        res = torch.bfloat16 if case["res"] == "bf16" else torch.float32
        s["eps"], s["scale"] = 1e-5, 0.75
        s["y"] = _randn(g, M, D, std=0.3)
        s["w_post"] = 1.0 + 0.1 * torch.randn(D, generator=g, device=DEVICE) if case["post"] else None
        s["gate"] = 0.5 + 0.2 * torch.randn(D, generator=g, device=DEVICE) if case["gate"] else None
        s["w_pre"] = 1.0 + 0.1 * torch.randn(D, generator=g, device=DEVICE)
        s["h"] = _randn(g, M, D, std=2.0, dtype=res)
        if op == "norm_bwd":
            h_out, _, s["rstd_post"], s["rstd_pre"] = _norm_forward(s, torch.float32)
            s["h_out"] = h_out.to(res)
            s["dh_out"], s["dx"] = _randn(g, M, D, std=0.1, dtype=res), _randn(g, M, D, std=0.1)
            del s["h"]
    else:
        M, V, ld = case["M"], case["V"], case["ld"]
        rows = torch.zeros((M, ld), device=DEVICE, dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        for i in range(0, M, 512):  # in pieces: the fp32 samples of a large case need not exist at once
            rows[i:i + 512, :V] = torch.randn((min(512, M - i), V), generator=g, device=DEVICE) * 2.5
        s["logits"] = rows[:, :V]
        s["targets"] = torch.randint(0, V, (M,), generator=g, device=DEVICE)
        # The targets are likely tokens, the last few ids are masked out, some positions are not scored.
        s["logits"].scatter_add_(1, s["targets"][:, None],
                                 torch.full((M, 1), 6.0, device=DEVICE, dtype=rows.dtype))
        if V > 1000:
            masked = torch.arange(V - 16, V, device=DEVICE)
            s["logits"][:, V - 16:] = float("-inf")
            s["targets"] = torch.where(torch.isin(s["targets"], masked), 0, s["targets"])
        if M > 8:
            s["targets"][::9] = -100
        s["inv_temp"] = 1.0 / case["temp"]
        if op == "logp_bwd":
            _, s["entropy"], s["row_max"], s["log_sum"] = _logp_forward(s, torch.float32)
            s["g_logp"] = -torch.rand(M, generator=g, device=DEVICE) / M
            s["g_entropy"] = -0.01 * torch.rand(M, generator=g, device=DEVICE) / M
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _weight(s, N, K):
    """The dequantized 4-bit weight: bf16(L[code] a) with a = fp32(fp32(q / 127 c2) + mu)."""
    codes = torch.stack((s["packed"] & 15, s["packed"] >> 4), 1).view(-1).long()
    chunk = torch.arange(N * K // BLOCK, device=DEVICE) // 256
    a = s["qscale"].float() / 127.0 * s["c2"][chunk] + s["mu"]
    w = torch.tensor(NF4, device=DEVICE)[codes].view(-1, BLOCK) * a[:, None]
    return w.to(torch.bfloat16).float().view(N, K)


def _norm_forward(s, dtype):
    """(h', x, rstd of y, rstd of h') in `dtype`; x is the norm of h' before that is rounded for storage."""
    y = s["y"].to(dtype)
    rstd_post = None
    if s["w_post"] is not None:
        rstd_post = 1.0 / torch.sqrt((y * y).mean(1) + s["eps"])
        y = y * rstd_post[:, None] * s["w_post"].to(dtype)
    if s["gate"] is not None:
        y = y * s["gate"].to(dtype)
    h_out = s["h"].to(dtype) + s["scale"] * y
    rstd_pre = 1.0 / torch.sqrt((h_out * h_out).mean(1) + s["eps"])
    return h_out, h_out * rstd_pre[:, None] * s["w_pre"].to(dtype), rstd_post, rstd_pre


def _norm_backward(s, dtype):
    h, rstd = s["h_out"].to(dtype), s["rstd_pre"].to(dtype)[:, None]
    dx, n = s["dx"].to(dtype), h * rstd
    dn = dx * s["w_pre"].to(dtype)
    g = s["dh_out"].to(dtype) + rstd * (dn - n * (dn * n).mean(1, keepdim=True))
    out = {"dh": g.to(s["h_out"].dtype), "dw_pre": (dx * n).sum(0)}
    y, dp = s["y"].to(dtype), s["scale"] * g
    p = y
    if s["w_post"] is not None:
        rstd = s["rstd_post"].to(dtype)[:, None]
        n = y * rstd
        p = n * s["w_post"].to(dtype)
    if s["gate"] is not None:
        out["dgate"] = (dp * p).sum(0)
        dp = dp * s["gate"].to(dtype)
    if s["w_post"] is not None:
        out["dw_post"] = (dp * n).sum(0)
        dn = dp * s["w_post"].to(dtype)
        dp = rstd * (dn - n * (dn * n).mean(1, keepdim=True))
    out["dy"] = dp.to(torch.bfloat16)
    return out


def _logp_forward(s, dtype):
    """(log probability of each target, entropy, row maximum, log of the sum relative to it)."""
    x = s["logits"].to(dtype)
    row_max = x.amax(1)
    d = (x - row_max[:, None]) * s["inv_temp"]
    e = torch.exp(d)
    total = e.sum(1)
    log_sum = torch.log(total)
    entropy = log_sum - torch.where(e > 0, e * d, torch.zeros_like(e)).sum(1) / total
    t = s["targets"]
    logp = d.gather(1, t.clamp(min=0)[:, None])[:, 0] - log_sum
    return torch.where(t >= 0, logp, torch.zeros_like(logp)), entropy, row_max, log_sum


def _logp_top(s, k, row_max, log_sum, dtype):
    """The k largest logits of each row (the lowest id first among equals) and their log probabilities."""
    values, ids = torch.sort(s["logits"], dim=1, descending=True, stable=True)
    values, ids = values[:, :k].to(dtype), ids[:, :k]
    return ids.to(torch.int32), (values - row_max[:, None]) * s["inv_temp"] - log_sum[:, None]


def _logp_backward(s, dtype):
    d = (s["logits"].to(dtype) - s["row_max"].to(dtype)[:, None]) * s["inv_temp"] - s["log_sum"].to(dtype)[:, None]
    p = torch.exp(d)
    scored = (s["targets"] >= 0).to(dtype)
    g = (s["g_logp"].to(dtype) * scored)[:, None]
    spread = torch.where(p > 0, p * (d + s["entropy"].to(dtype)[:, None]), torch.zeros_like(p))
    grad = -g * p - s["g_entropy"].to(dtype)[:, None] * spread
    grad.scatter_add_(1, s["targets"].clamp(min=0)[:, None], g)
    return (grad * s["inv_temp"]).to(s["logits"].dtype)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "ckpt":
        codes, step = _checkpoint(s["x"], c["fmt"])
        return {"values": _checkpoint_values(codes, step, c["fmt"]).to(torch.bfloat16), "step": step}
    if op == "linear":
        x = _checkpoint_values(s["codes"], s["step"], c["fmt"])
        dy, A, B = s["dy"].float(), s["A"].float(), s["B"].float()
        u = s["u"] if s["u"] is not None else x @ A.t()
        v = dy @ B
        out = {"dA": s["scale"] * (v.t() @ x), "dB": s["scale"] * (dy.t() @ u)}
        if c["dx"]:
            out["dX"] = (dy @ _weight(s, c["N"], c["K"]) + s["scale"] * (v @ A)).to(torch.bfloat16)
        return out
    if op == "norm_fwd":
        h_out, x, rstd_post, rstd_pre = _norm_forward(s, torch.float32)
        out = {"h_out": h_out.to(s["h"].dtype), "x": x.to(torch.bfloat16), "rstd_pre": rstd_pre}
        if c["post"]:
            out["rstd_post"] = rstd_post
        if c["ckpt"]:
            codes, out["step"] = _checkpoint(out["x"], "e4m3")
            out["codes"] = codes.view(torch.float8_e4m3fn)
        return out
    if op == "norm_bwd":
        return _norm_backward(s, torch.float32)
    if op == "logp_fwd":
        logp, entropy, row_max, log_sum = _logp_forward(s, torch.float32)
        out = {"logp": logp, "entropy": entropy, "row_max": row_max, "log_sum": log_sum}
        if c["top"]:
            out["top_ids"], out["top_logp"] = _logp_top(s, c["top"], row_max, log_sum, torch.float32)
        return out
    return {"dlogits": _logp_backward(s, torch.float32)}


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _buffers(s):
    """Output buffers, descriptors and workspace, made on a state's first pass and kept, as a program keeps them."""
    from bit_nf4_quantized_blk_b200 import binding as q

    c = s["case"]
    op, f32 = c["op"], torch.float32
    b = {"q": q}
    fmt = q.ACT8_INT8 if c.get("fmt") == "int8" else q.ACT8_E4M3
    if op == "ckpt":
        b["act"] = q.Act8.empty(c["M"], c["K"], fmt=fmt)
        b["values"] = torch.empty_like(s["x"])
    elif op == "linear":
        M, N, K, r = (c[k] for k in ("M", "N", "K", "r"))
        b["w"] = q.NF4Weight(N, K, s["packed"], s["qscale"], s["c2"], s["mu"])
        b["act"] = q.Act8(M, K, s["codes"], s["step"], fmt)
        b["ws"] = torch.empty(q.qlora_linear_ws_bytes(M, N, K, r), dtype=torch.uint8, device=DEVICE)
        q.qlora_workspace_reset(b["ws"])
        b["dX"] = torch.empty((M, K), dtype=torch.bfloat16, device=DEVICE) if c["dx"] else None
        b["dA"] = torch.empty((r, K), dtype=f32, device=DEVICE)
        b["dB"] = torch.empty((N, r), dtype=f32, device=DEVICE)
    elif op == "norm_fwd":
        M, D = c["M"], c["D"]
        b["h_out"], b["x"] = torch.empty_like(s["h"]), torch.empty((M, D), dtype=torch.bfloat16, device=DEVICE)
        b["act"] = q.Act8.empty(M, D, fmt=q.ACT8_E4M3) if c["ckpt"] else None
        b["rstd_post"] = torch.empty(M, dtype=f32, device=DEVICE) if c["post"] else None
        b["rstd_pre"] = torch.empty(M, dtype=f32, device=DEVICE)
    elif op == "norm_bwd":
        M, D = c["M"], c["D"]
        b["ws"] = torch.empty(q.qlora_residual_norm_ws_bytes(M, D), dtype=torch.uint8, device=DEVICE)
        b["dh"], b["dy"] = torch.empty_like(s["h_out"]), torch.empty_like(s["y"])
        b["dw_post"] = torch.empty(D, dtype=f32, device=DEVICE) if c["post"] else None
        b["dgate"] = torch.empty(D, dtype=f32, device=DEVICE) if c["gate"] else None
        b["dw_pre"] = torch.empty(D, dtype=f32, device=DEVICE)
    elif op == "logp_fwd":
        M, k = c["M"], c["top"]
        for name in ("logp", "entropy", "row_max", "log_sum"):
            b[name] = torch.empty(M, dtype=f32, device=DEVICE)
        b["top_ids"] = torch.empty((M, k), dtype=torch.int32, device=DEVICE) if k else None
        b["top_logp"] = torch.empty((M, k), dtype=f32, device=DEVICE) if k else None
    else:
        b["dlogits"] = torch.empty((c["M"], c["ld"]), dtype=s["logits"].dtype, device=DEVICE)[:, :c["V"]]
    return b


def _own(s):
    if "buffers" not in s:
        s["buffers"] = _buffers(s)
    b, c = s["buffers"], s["case"]
    q, op = b["q"], c["op"]
    if op == "ckpt":
        q.qlora_act8_quantize(s["x"], b["act"])
        q.qlora_act8_dequantize(b["act"], b["values"])
        return {"values": b["values"], "step": b["act"].step.view(c["M"], -1)}
    if op == "linear":
        q.qlora_linear_bwd_act8(b["w"], b["act"], s["dy"], s["A"], s["B"], c["r"], s["scale"], b["dX"], 0, b["dA"],
                                b["dB"], b["ws"], U=s["u"])
        return {k: b[k] for k in ("dA", "dB") + (("dX",) if c["dx"] else ())}
    if op == "norm_fwd":
        q.qlora_residual_norm_fwd(s["h"], s["y"], s["w_post"], s["gate"], s["scale"], s["w_pre"], s["eps"],
                                  b["h_out"], b["x"], b["act"], b["rstd_post"], b["rstd_pre"])
        out = {k: b[k] for k in ("h_out", "x", "rstd_pre") + (("rstd_post",) if c["post"] else ())}
        if c["ckpt"]:
            out["step"] = b["act"].step.view(c["M"], -1)
            out["codes"] = b["act"].codes.view(torch.float8_e4m3fn).view(c["M"], -1)
        return out
    if op == "norm_bwd":
        q.qlora_residual_norm_bwd(s["dh_out"], s["dx"], s["h_out"], s["y"], s["w_post"], s["gate"], s["scale"],
                                  s["w_pre"], s.get("rstd_post"), s["rstd_pre"], b["dh"], b["dy"], b["dw_post"],
                                  b["dgate"], b["dw_pre"], b["ws"])
        return {k: b[k] for k in ("dh", "dy", "dw_post", "dgate", "dw_pre") if b[k] is not None}
    if op == "logp_fwd":
        q.qlora_token_logprobs_fwd(s["logits"], s["targets"], s["inv_temp"], b["logp"], b["entropy"], b["row_max"],
                                   b["log_sum"], c["top"], b["top_ids"], b["top_logp"])
        names = ("logp", "entropy", "row_max", "log_sum") + (("top_ids", "top_logp") if c["top"] else ())
        return {k: b[k] for k in names}
    q.qlora_token_logprobs_bwd(s["logits"], s["targets"], s["inv_temp"], s["row_max"], s["log_sum"], s["entropy"],
                               s["g_logp"], s["g_entropy"], b["dlogits"])
    return {"dlogits": b["dlogits"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# What a case cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "ckpt":  # X in, the checkpoint out and in again, its values out
        n = case["M"] * case["K"]
        return {"bytes": 4 * n + 2 * (n + 2 * n // BLOCK), "flops": 6 * n}
    if op == "linear":
        M, N, K, r = (case[k] for k in ("M", "N", "K", "r"))
        b = M * K * (1 + 2 / BLOCK) + 2 * M * N + 2 * r * (N + K) + 4 * r * (N + K) + (4 * M * r if case["saved_u"] else 0)
        f = 2 * M * r * (2 * N + K + (0 if case["saved_u"] else K))
        if case["dx"]:
            b += N * K * (0.5 + 1 / BLOCK) + N * K / (256 * BLOCK) * 4 + 2 * M * K
            f += 2 * M * K * (N + r)
        return {"bytes": int(b), "flops": f}
    if op in ("norm_fwd", "norm_bwd"):
        M, D, res = case["M"], case["D"], 2 if case["res"] == "bf16" else 4
        params = 4 * D * (1 + case["post"] + case["gate"])
        if op == "norm_fwd":
            b = M * D * (2 * res + 4) + params + 4 * M * (1 + case["post"])
            b += M * D * (1 + 2 / BLOCK) if case["ckpt"] else 0
            return {"bytes": int(b), "flops": M * D * 12}
        return {"bytes": M * D * (3 * res + 6) + 2 * params + 4 * M * (1 + case["post"]), "flops": M * D * 24}
    n = case["M"] * case["V"]
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "logp_fwd":
        return {"bytes": n * size + case["M"] * (24 + 8 * case["top"]), "flops": 6 * n}
    return {"bytes": 2 * n * size + case["M"] * 28, "flops": 8 * n}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_bf16(v):
    """Round 64-bit values to bf16 (8 significant bits, ties to even); the cases hold no subnormals."""
    m, e = torch.frexp(v)
    return torch.ldexp(torch.round(m * 256.0) / 256.0, e)


def _exact_codes(x, fmt):
    """(code values, steps) of the rows' blocks in 64 bits."""
    v = x.double().reshape(-1, BLOCK)
    step = _exact_bf16(v.abs().max(1, keepdim=True).values / (127.0 if fmt == "int8" else 256.0))
    q = torch.nan_to_num(v / step, nan=0.0)  # 0 / 0 in a block of zeros
    if fmt == "int8":
        return torch.round(q), step
    _, e = torch.frexp(q)
    unit = torch.ldexp(torch.ones_like(q), e.clamp(min=-5) - 4)  # 4 significant bits, down to 2^-9
    return torch.round(q / unit) * unit, step


def _exact_linear(s, c):
    N, K, r = c["N"], c["K"], c["r"]
    M = c["M"]
    q = s["codes"].view(torch.int8 if c["fmt"] == "int8" else torch.float8_e4m3fn).double().view(-1, BLOCK)
    x = _exact_bf16(q * s["step"].double().view(-1, 1)).view(M, K)
    A, B, dy = s["A"].double(), s["B"].double(), s["dy"].double()
    v = dy.matmul(B)
    u = s["u"].double() if s["u"] is not None else x.matmul(A.t())
    out = {"dA": s["scale"] * v.t().matmul(x), "dB": s["scale"] * dy.t().matmul(u)}
    del x, u
    if c["dx"]:
        # The block scale is two fp32 operations by definition, the weight their product rounded to bf16.
        a = (s["qscale"].float() / 127.0) * s["c2"].repeat_interleave(256)[: N * K // BLOCK] + s["mu"]
        level = torch.tensor(NF4, dtype=torch.float64, device=DEVICE)
        w = torch.empty((N * K // 2, 2), dtype=torch.float64, device=DEVICE)
        w[:, 0], w[:, 1] = level[(s["packed"] % 16).long()], level[(s["packed"] // 16).long()]
        w = _exact_bf16((w.view(-1, BLOCK) * a.double()[:, None]).float().double()).view(N, K)
        out["dX"] = dy.matmul(w) + s["scale"] * v.matmul(A)
    return out


def _exact_norm_forward(s, c):
    y, h = s["y"].double(), s["h"].double()
    D, out = c["D"], {}
    if c["post"]:
        out["rstd_post"] = (y.square().sum(1) / D + s["eps"]).rsqrt()
        y = torch.einsum("md,m,d->md", y, out["rstd_post"], s["w_post"].double())
    if c["gate"]:
        y = y * s["gate"].double()
    total = h + y * s["scale"]
    out["h_out"] = total
    out["rstd_pre"] = (total.square().sum(1) / D + s["eps"]).rsqrt()
    out["x"] = torch.einsum("md,m,d->md", total, out["rstd_pre"], s["w_pre"].double())
    if c["ckpt"]:
        q, step = _exact_codes(_exact_bf16(out["x"]), "e4m3")
        out["codes"], out["step"] = q.view(c["M"], D), step.view(c["M"], -1)
    return out


def _exact_norm_backward(s, c):
    """By the derivative of each formula: d(v rstd)/dv = rstd (1 - n n^T / D)."""
    D, out = c["D"], {}
    h, dx = s["h_out"].double(), s["dx"].double()
    r1 = s["rstd_pre"].double().unsqueeze(1)
    out["dw_pre"] = torch.einsum("md,md->d", dx, h * r1)
    t = dx * s["w_pre"].double()
    g = s["dh_out"].double() + r1 * t - h * r1.pow(3) * ((t * h).sum(1, keepdim=True) / D)
    out["dh"] = g
    y = s["y"].double()
    r2 = s["rstd_post"].double().unsqueeze(1) if c["post"] else 1.0
    wp = s["w_post"].double() if c["post"] else 1.0
    gt = s["gate"].double() if c["gate"] else 1.0
    if c["gate"]:
        out["dgate"] = s["scale"] * (g * y * r2 * wp).sum(0)
    if c["post"]:
        out["dw_post"] = s["scale"] * (g * gt * y * r2).sum(0)
        t = s["scale"] * g * gt * wp
        out["dy"] = r2 * t - y * r2.pow(3) * ((t * y).sum(1, keepdim=True) / D)
    else:
        out["dy"] = s["scale"] * g * gt
    return out


def _exact_logp(s, c):
    out = []
    it = s["inv_temp"]
    step = max(1, (1 << 26) // c["V"])
    for i in range(0, c["M"], step):  # rows in pieces: 64-bit copies of a large case need not exist at once
        z = s["logits"][i:i + step].double() * it
        t = s["targets"][i:i + step]
        logp = torch.log_softmax(z, 1)
        p = logp.exp()
        plogp = torch.nan_to_num(p * logp, nan=0.0)  # 0 log 0
        at = logp.gather(1, t.clamp(min=0).unsqueeze(1)).squeeze(1)
        if c["op"] == "logp_fwd":
            top = z.max(1).values
            row = {"logp": torch.where(t < 0, 0.0, at), "entropy": -plogp.sum(1), "row_max": top / it,
                   "log_sum": torch.logsumexp(z, 1) - top}
            if c["top"]:
                # Ids by value, then by position: a 64-bit key of both.
                order = torch.argsort(z, dim=1, descending=True, stable=True)[:, : c["top"]]
                row["top_ids"], row["top_logp"] = order.to(torch.int32), logp.gather(1, order)
        else:
            H = -plogp.sum(1, keepdim=True)
            g = torch.where(t < 0, 0.0, s["g_logp"][i:i + step].double()).unsqueeze(1)
            gh = s["g_entropy"][i:i + step].double().unsqueeze(1)
            grad = -(g * p) - gh * (plogp + p * H)
            grad.scatter_add_(1, t.clamp(min=0).unsqueeze(1), g)
            row = {"dlogits": grad * it}
        out.append(row)
    return {k: torch.cat([r[k] for r in out]) for k in out[0]}


def exact(case, seed):
    s, c = prepare(case, seed), dict(case)
    op = c["op"]
    if op == "ckpt":
        q, step = _exact_codes(s["x"], c["fmt"])
        return {"values": _exact_bf16(q * step).view(c["M"], c["K"]), "step": step.view(c["M"], -1)}
    if op == "linear":
        return _exact_linear(s, c)
    if op == "norm_fwd":
        return _exact_norm_forward(s, c)
    if op == "norm_bwd":
        return _exact_norm_backward(s, c)
    return _exact_logp(s, c)
