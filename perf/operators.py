"""The operators around the FP8 linear layer, as cases to measure.

Four calls, two operators with their gradients:

- ``linear``: the block-scaled FP8 product with bias, activation and residual
  in its epilogue, the activation operand as E4M3 codes or as bf16 quantized
  in the call (few rows);
- ``linear_backward``: from the incoming gradient and the kept pre-activation
  to the E4M3 operands of the two backward products and the bias gradient;
- ``xent``: the bf16 head's product with the softmax cross entropy of its
  logits, which are never stored;
- ``xent_backward``: its gradients for the hidden states and the head's weight.

``run`` computes a case in plain torch operations (``own`` false) or calls
the library (``own`` true).
"""

import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
SCALE_FLOOR = 2.0 ** -64
IGNORE = -100
GELU_C = math.sqrt(2.0 / math.pi)


# ----------------------------------------------------------------------------
# cases


def listed():
    return [
        # the FP8 linear layer of one decoded token (the activation arrives in
        # bf16): the weight's stream and the call's latency
        {"name": "linear_token", "op": "linear", "M": 1, "N": 18432, "K": 7168, "a": "bf16",
         "act": "silu", "bias": True, "residual": False, "z": False},
        # the up projection of a dense training step; the pre-activation is
        # kept for the backward pass
        {"name": "linear_up", "op": "linear", "M": 4096, "N": 18432, "K": 7168, "a": "e4m3",
         "act": "gelu", "bias": True, "residual": False, "z": True},
        # its down projection, added to the residual stream
        {"name": "linear_down", "op": "linear", "M": 4096, "N": 7168, "K": 18432, "a": "e4m3",
         "act": "none", "bias": True, "residual": True, "z": False},
        # ragged rows and columns, every part of the epilogue at once
        {"name": "linear_odd", "op": "linear", "M": 333, "N": 2050, "K": 2048, "a": "e4m3",
         "act": "silu", "bias": True, "residual": True, "z": True},
        # backward of linear_up's epilogue
        {"name": "linear_grad", "op": "linear_backward", "M": 4096, "N": 18432, "act": "gelu"},
        # few ragged tokens, where the launches count
        {"name": "linear_grad_odd", "op": "linear_backward", "M": 333, "N": 2048, "act": "silu"},
        # scoring one token over a large vocabulary: the head weight's stream
        {"name": "xent_token", "op": "xent", "M": 1, "V": 129280, "K": 7168, "ignored": 0.0},
        # a batch of short answers being scored, small head, prompt masked
        {"name": "xent_odd", "op": "xent", "M": 1531, "V": 32003, "K": 2048, "ignored": 0.6},
        # the loss of a training step
        {"name": "xent_train", "op": "xent", "M": 4096, "V": 129280, "K": 7168, "ignored": 0.0},
        # a tiny head: latency
        {"name": "xent_grad_small", "op": "xent_backward", "M": 130, "V": 1003, "K": 512,
         "ignored": 0.1},
        # tuning on answers alone: most positions carry no loss
        {"name": "xent_grad_odd", "op": "xent_backward", "M": 1531, "V": 32003, "K": 2048,
         "ignored": 0.6},
        # the gradients of a training step
        {"name": "xent_grad_train", "op": "xent_backward", "M": 4096, "V": 129280, "K": 7168,
         "ignored": 0.0},
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n if n != 3072 else n + 1


def _log128(rng, lo, hi):
    n = max(1, round(_log(rng, lo, hi) / 128)) * 128
    return n if n != 3072 else n + 128


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "xent", "xent_backward"])
    if op == "linear":
        M, N = _log(rng, 1, 4096), _log(rng, 100, 18432)
        a = "bf16" if M <= 64 and rng.random() < 0.5 else "e4m3"
        return {"op": op, "M": M, "N": N, "K": _log128(rng, 512, 7168), "a": a,
                "act": rng.choice(["none", "relu", "silu", "gelu"]),
                "bias": rng.random() < 0.7, "residual": rng.random() < 0.5,
                "z": rng.random() < 0.5}
    if op == "linear_backward":
        return {"op": op, "M": _log(rng, 30, 4096), "N": _log128(rng, 512, 18432),
                "act": rng.choice(["none", "relu", "silu", "gelu"])}
    if op == "xent":
        return {"op": op, "M": _log(rng, 1, 4096), "V": _log(rng, 1000, 129280),
                "K": _log128(rng, 512, 7168), "ignored": rng.choice([0.0, 0.1, 0.5])}
    return {"op": op, "M": _log(rng, 60, 4096), "V": _log(rng, 1000, 129280),
            "K": _log128(rng, 512, 7168), "ignored": rng.choice([0.0, 0.1, 0.5])}


def _valid(case):
    return case["M"] - int(case["M"] * case["ignored"])


def work(case):
    M, op = case["M"], case["op"]
    if op == "linear":
        N, K = case["N"], case["K"]
        a = M * K * (2 if case["a"] == "bf16" else 1) + (0 if case["a"] == "bf16" else M * K // 32)
        nbytes = a + N * K + 4 * (-(-N // 128)) * (K // 128) + 2 * M * N
        nbytes += (4 * N if case["bias"] else 0) + (2 * M * N if case["residual"] else 0)
        nbytes += 2 * M * N if case["z"] else 0
        return {"bytes": nbytes, "flops": 2 * M * N * K}
    if op == "linear_backward":
        N = case["N"]
        mp = -(-M // 128) * 128
        nbytes = 4 * M * N + M * N + mp * N + 4 * M * (N // 128) + 4 * (mp // 128) * N + 4 * N
        return {"bytes": nbytes, "flops": 20 * M * N}
    V, K, mv = case["V"], case["K"], _valid(case)
    if op == "xent":
        return {"bytes": 2 * mv * K + 2 * V * K + 16 * M, "flops": 2 * mv * V * K}
    # the logits are not kept: they are rebuilt, then two products
    return {"bytes": 2 * mv * K + 2 * V * K + 16 * M + 2 * M * K + 2 * V * K,
            "flops": 6 * mv * V * K}


# ----------------------------------------------------------------------------
# inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _activation(g, M, K):
    """Rows of different size and 0.1% outliers, as hidden states have."""
    x = _randn(g, M, K) * torch.exp(_randn(g, M, 1))
    far = torch.rand(M, K, generator=g, device=DEV) < 1e-3
    return torch.where(far, 20.0 * x, x).to(torch.bfloat16)


def _quant_tiles(x):
    """bf16 or fp32 [M][K] -> E4M3 values fp32, scales [K/128][M] (online 1x128)."""
    M, K = x.shape
    t = x.float().view(M, K // 128, 128)
    a = t.abs().amax(dim=2).clamp_min(SCALE_FLOOR)
    q = (t * (E4M3_MAX / a)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(M, K), (a / E4M3_MAX).t().contiguous()


def _quant_blocks(w):
    """fp32 [N][K] -> E4M3 codes, scales [ceil(N/128)][K/128] (online 128x128)."""
    N, K = w.shape
    nb = -(-N // 128)
    t = torch.nn.functional.pad(w, (0, 0, 0, nb * 128 - N)).view(nb, 128, K // 128, 128)
    a = t.abs().amax(dim=(1, 3)).clamp_min(SCALE_FLOOR)
    q = (t * (E4M3_MAX / a)[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    q = q.to(torch.float8_e4m3fn).view(nb * 128, K)[:N].contiguous()
    return q, (a / E4M3_MAX).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    M, op = case["M"], case["op"]
    if op == "linear":
        N, K = case["N"], case["K"]
        x = _activation(g, M, K)
        if case["a"] == "bf16":
            s["x"], s["sx"] = x, None
        else:
            q, sx = _quant_tiles(x)
            s["x"], s["sx"] = q.view(torch.uint8), sx
        # 1/sqrt(K) of the row's size: pre-activations of order one
        q, sw = _quant_blocks(_randn(g, N, K) / math.sqrt(K))
        s["w"], s["sw"] = q.view(torch.uint8), sw
        s["b"] = 0.1 * _randn(g, N) if case["bias"] else None
        s["r"] = _randn(g, M, N).to(torch.bfloat16) if case["residual"] else None
        return s
    if op == "linear_backward":
        N = case["N"]
        s["dy"] = (1e-3 * _randn(g, M, N) * torch.exp(_randn(g, M, 1))).to(torch.bfloat16)
        s["zk"] = (1.5 * _randn(g, M, N)).to(torch.bfloat16)
        return s
    V, K = case["V"], case["K"]
    s["x"] = _randn(g, M, K).to(torch.bfloat16)
    # logits of standard deviation 1.5
    s["w"] = (_randn(g, V, K) * (1.5 / math.sqrt(K))).to(torch.bfloat16)
    t = torch.randint(V, (M,), generator=g, device=DEV)
    skip = torch.randperm(M, generator=g, device=DEV)[:M - _valid(case)]
    t[skip] = IGNORE
    s["t"] = t
    if op == "xent_backward":
        # what the forward pass left, and the gradient of the mean loss
        s["lse"] = torch.cat([torch.logsumexp(_mm(c, s["w"]), dim=1)
                              for c in s["x"].split(1024)])
        s["lse"][t == IGNORE] = 0.0
        s["dloss"] = torch.full((M,), 1.0 / max(1, _valid(case)), device=DEV)
    return s


def _mm(a, b):
    """a . b^T in 32 bits."""
    return torch.mm(a.float(), b.float().t())


# ----------------------------------------------------------------------------
# plain forms


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.tanh(GELU_C * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        t = torch.tanh(GELU_C * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * GELU_C * (1.0 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain_linear(s):
    M, N, K = s["M"], s["N"], s["K"]
    if s["sx"] is None:
        q, sx = _quant_tiles(s["x"])
    else:
        q, sx = s["x"].view(torch.float8_e4m3fn), s["sx"]
    a = (q.float().view(M, K // 128, 128) * sx.t()[:, :, None]).view(M, K)
    sw = s["sw"].repeat_interleave(128, dim=0)[:N]
    b = (s["w"].view(torch.float8_e4m3fn).float().view(N, K // 128, 128) * sw[:, :, None])
    z = torch.mm(a, b.view(N, K).t())
    if s["b"] is not None:
        z = z + s["b"]
    y = _act(z, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.to(torch.bfloat16), "z": z.to(torch.bfloat16) if s["z"] else None}


def _plain_linear_backward(s):
    M, N = s["M"], s["N"]
    dz = s["dy"].float() * _act_grad(s["zk"].float(), s["act"])
    q, sq = _quant_tiles(dz)
    mp = -(-M // 128) * 128
    qt, st = _quant_tiles(torch.nn.functional.pad(dz, (0, 0, 0, mp - M)).t().contiguous())
    return {"q": q, "s": sq, "qt": qt, "st": st, "db": dz.sum(dim=0)}


def _plain_xent(s):
    w = s["w"].float()
    keep = s["t"] != IGNORE
    l = torch.mm(s["x"].float(), w.t())
    m = l.amax(dim=1)
    lse = m + torch.log(torch.exp(l - m[:, None]).sum(dim=1))
    at = l.gather(1, s["t"].clamp_min(0)[:, None])[:, 0]
    zero = torch.zeros_like(lse)
    return {"loss": torch.where(keep, lse - at, zero), "lse": torch.where(keep, lse, zero)}


def _plain_xent_backward(s):
    x, w = s["x"].float(), s["w"].float()
    keep = s["t"] != IGNORE
    g = torch.exp(torch.mm(x, w.t()) - s["lse"][:, None])
    g.scatter_add_(1, s["t"].clamp_min(0)[:, None], torch.full_like(g[:, :1], -1.0))
    g *= torch.where(keep, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
    return {"dx": torch.mm(g, w).to(torch.bfloat16), "dw": torch.mm(g.t(), x).to(torch.bfloat16)}


# ----------------------------------------------------------------------------
# one pass


def run(s):
    if not own:
        return {"linear": _plain_linear, "linear_backward": _plain_linear_backward,
                "xent": _plain_xent, "xent_backward": _plain_xent_backward}[s["op"]](s)
    from fp8_block_scaled_05_amd import fp8bs
    if s["op"] == "linear":
        z = (torch.empty(s["M"], s["N"], dtype=torch.bfloat16, device=DEV) if s["z"] else None)
        y = fp8bs.fp8_block_gemm_epilogue(s["x"], s["sx"], s["w"], s["sw"], bias=s["b"],
                                          act=s["act"], residual=s["r"], z=z)
        return {"y": y, "z": z}
    if s["op"] == "linear_backward":
        q, sq, qt, st, db = fp8bs.fp8_quant_epilogue_backward(s["dy"], s["zk"], act=s["act"])
        return {"q": q.view(torch.float8_e4m3fn), "s": sq, "qt": qt.view(torch.float8_e4m3fn),
                "st": st, "db": db}
    if s["op"] == "xent":
        loss, lse = fp8bs.bf16_linear_xent(s["x"], s["w"], s["t"], ignore_index=IGNORE)
        return {"loss": loss, "lse": lse}
    dx, dw = fp8bs.bf16_linear_xent_backward(s["x"], s["w"], s["t"], s["lse"], s["dloss"],
                                             ignore_index=IGNORE)
    return {"dx": dx, "dw": dw}


# ----------------------------------------------------------------------------
# the definitions in 64 bits


def _exact_codes(x64, dim_tiles):
    """1x128 tiles of fp64 [R][C] along C: (codes, scales [C/128][R]) with the
    format's own fp32 scale and reciprocal."""
    R, C = x64.shape
    t = x64.reshape(R, dim_tiles, C // dim_tiles)
    a = t.abs().amax(dim=2).clamp_min(SCALE_FLOOR)
    v = (t * (E4M3_MAX / a)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    # nearest E4M3 value, ties to even, straight from the format: 3 mantissa
    # bits, smallest exponent -6
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -20))).clamp_min(-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(v / step) * step).reshape(R, C), (a / E4M3_MAX).t().contiguous()


def exact(case, seed):
    s = prepare(case, seed)
    M, op = case["M"], case["op"]
    f64 = torch.float64
    if op == "linear":
        N, K = case["N"], case["K"]
        a = torch.empty(M, K, dtype=f64, device=DEV)
        b = torch.empty(N, K, dtype=f64, device=DEV)
        for kb in range(K // 128):
            c = slice(128 * kb, 128 * kb + 128)
            if s["sx"] is None:
                # the codes are defined by fp32 scale and reciprocal
                t = s["x"][:, c].float()
                am = torch.maximum(t.abs().amax(dim=1), torch.tensor(SCALE_FLOOR, device=DEV))
                v = (t * (E4M3_MAX / am)[:, None]).to(f64)
                e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -20))).clamp_min(-6.0)
                step = torch.exp2(e - 3.0)
                v = (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
                a[:, c] = v * (am / E4M3_MAX).to(f64)[:, None]
            else:
                a[:, c] = s["x"][:, c].view(torch.float8_e4m3fn).to(f64) * s["sx"][kb].to(f64)[:, None]
            rows = s["sw"][:, kb].to(f64)[torch.arange(N, device=DEV) // 128]
            b[:, c] = s["w"][:, c].view(torch.float8_e4m3fn).to(f64) * rows[:, None]
        z = a @ b.T
        if s["b"] is not None:
            z += s["b"].to(f64)
        act = case["act"]
        if act == "silu":
            y = z * torch.sigmoid(z)
        elif act == "gelu":
            y = torch.nn.functional.gelu(z, approximate="tanh")
        else:
            y = torch.relu(z) if act == "relu" else z.clone()
        if s["r"] is not None:
            y += s["r"].to(f64)
        return {"y": y, "z": z if case["z"] else None}
    if op == "linear_backward":
        N = case["N"]
        z = s["zk"].to(f64)
        act = case["act"]
        if act == "silu":
            d = torch.sigmoid(z) * (1 + z * torch.sigmoid(-z))
        elif act == "gelu":
            u = GELU_C * (z + 0.044715 * z ** 3)
            d = torch.sigmoid(2 * u) + z * GELU_C * (1 + 0.134145 * z ** 2) / (2 * torch.cosh(u) ** 2)
        else:
            d = (z > 0).to(f64) if act == "relu" else torch.ones_like(z)
        dz = s["dy"].to(f64) * d
        mp = -(-M // 128) * 128
        dzt = torch.zeros(N, mp, dtype=f64, device=DEV)
        dzt[:, :M] = dz.T
        q, sq = _exact_codes(dz, N // 128)
        qt, st = _exact_codes(dzt, mp // 128)
        return {"q": q, "s": sq, "qt": qt, "st": st, "db": dz.sum(dim=0)}
    V = case["V"]
    keep = torch.nonzero(s["t"] != IGNORE)[:, 0]
    x, w, t = s["x"][keep].to(f64), s["w"].to(f64), s["t"][keep]
    l = x @ w.T
    at = torch.arange(keep.numel(), device=DEV)
    if op == "xent":
        loss = torch.zeros(M, dtype=f64, device=DEV)
        lse = torch.zeros(M, dtype=f64, device=DEV)
        r = torch.logsumexp(l, dim=1)
        loss[keep], lse[keep] = r - l[at, t], r
        return {"loss": loss, "lse": lse}
    l -= s["lse"][keep].to(f64)[:, None]
    p = l.exp_()
    p[at, t] -= 1.0
    p *= s["dloss"][keep].to(f64)[:, None]
    dx = torch.zeros(M, case["K"], dtype=f64, device=DEV)
    dx[keep] = p @ w
    return {"dx": dx, "dw": p.T @ x}
