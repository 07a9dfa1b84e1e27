"""One training step of a small FP8 language model, from the embedding to the
updated weights, on the library's calls:

- residual MLP blocks ``y = x + W2 act(W1 x + b1) + b2`` with FP8 products: the
  up projection's epilogue applies bias and activation, keeps the
  pre-activation and emits the down projection's E4M3 input; the down
  projection's adds bias and residual;
- or, with ``block="gated"``, pre-norm gated blocks ``y = x + W2 (act(Wg n) *
  (Wu n))``, ``n = norm(x)``: the norm adds the residual and emits the E4M3 input
  of the gated product, which keeps gate and up and emits the down projection's;
  a last norm stands before the head;
- a bf16 head whose cross entropy never stores the logits, and its gradients;
- backward: the epilogues' backward emits the E4M3 operands of the FP8 data and
  weight gradients and the bias gradients; the data gradient's own epilogue
  adds the gradient that came along the residual.  The gated product's backward
  emits its operands and the down projection's in one pass, the norm's adds the
  gradient along the residual.

Embedding, the decoding of the kept activations and the Adam update are plain
torch.

Usage: ``python -m fp8_block_scaled_05_amd.train_step [--steps 60] [--block
gated]`` trains it to predict a fixed permutation of the vocabulary and prints
the losses.
"""

import argparse
from dataclasses import dataclass

import torch

from . import fp8bs


@dataclass(frozen=True)
class Config:
    vocab: int = 1000
    hidden: int = 256
    inner: int = 512
    layers: int = 2
    act: str = "gelu"
    block: str = "mlp"  # or "gated"


def init(cfg, seed=0, device="cuda"):
    """fp32 master weights."""
    g = torch.Generator(device=device).manual_seed(seed)

    def randn(*shape, std):
        return torch.randn(*shape, generator=g, device=device) * std

    p = {"embedding": randn(cfg.vocab, cfg.hidden, std=1.0),
         "head": randn(cfg.vocab, cfg.hidden, std=cfg.hidden ** -0.5)}
    if cfg.block not in ("mlp", "gated"):
        raise ValueError(f"block must be 'mlp' or 'gated', got {cfg.block!r}")
    if cfg.block == "gated":
        for i in range(cfg.layers):
            p[f"norm{i}"] = torch.ones(cfg.hidden, device=device)
            # the gate's rows, then the up projection's
            p[f"up{i}"] = randn(2 * cfg.inner, cfg.hidden, std=cfg.hidden ** -0.5)
            p[f"down{i}"] = randn(cfg.hidden, cfg.inner, std=cfg.inner ** -0.5)
        p["norm"] = torch.ones(cfg.hidden, device=device)
        return p
    for i in range(cfg.layers):
        p[f"up{i}"] = randn(cfg.inner, cfg.hidden, std=cfg.hidden ** -0.5)
        p[f"up_bias{i}"] = torch.zeros(cfg.inner, device=device)
        p[f"down{i}"] = randn(cfg.hidden, cfg.inner, std=cfg.inner ** -0.5)
        p[f"down_bias{i}"] = torch.zeros(cfg.hidden, device=device)
    return p


def _padded_rows(x):
    """Zero rows up to a multiple of 128 (the weight gradients' token groups)."""
    pad = -x.shape[0] % 128
    return torch.nn.functional.pad(x, (0, 0, 0, pad)) if pad else x


def _decode(q, s):
    """E4M3 codes [M][N] with scales [N/128][M] as bf16."""
    M, N = q.shape
    v = q.view(torch.float8_e4m3fn).float().view(M, N // 128, 128) * s[:, :M].t()[:, :, None]
    return v.view(M, N).to(torch.bfloat16)


def _weight_grad(qt, st, x):
    """dW = dz^T x from the gradient's token-grouped codes."""
    qx, sx = fp8bs.fp8_quant_act_128x1_t(_padded_rows(x))
    return fp8bs.fp8_block_gemm_rowscaled(qt, st, qx, sx)


def loss_and_grads(cfg, p, tokens, target, ignore_index=-100):
    """Mean loss over the positions that carry one, and the gradients of all
    weights (fp32 where the library gives fp32)."""
    bf16 = torch.bfloat16
    x = p["embedding"][tokens].to(bf16)
    if cfg.block == "gated":
        return _gated_loss_and_grads(cfg, p, tokens, x, target, ignore_index)
    kept = []
    for i in range(cfg.layers):
        qx, sx = fp8bs.fp8_quant_act_1x128(x)
        up = fp8bs.fp8_quant_w_128x128_t(p[f"up{i}"].to(bf16))
        down = fp8bs.fp8_quant_w_128x128_t(p[f"down{i}"].to(bf16))
        z = torch.empty(x.shape[0], cfg.inner, dtype=bf16, device=x.device)
        qh, sh = fp8bs.fp8_block_gemm_epilogue_e4m3_out(qx, sx, up[0], up[1],
                                                        bias=p[f"up_bias{i}"], act=cfg.act, z=z)
        y = fp8bs.fp8_block_gemm_epilogue(qh, sh, down[0], down[1], bias=p[f"down_bias{i}"],
                                          residual=x)
        kept.append((x, z, qh, sh, up, down))
        x = y
    grads = {}
    loss, dy, grads["head"] = _head(cfg, p, x, target, ignore_index)
    for i in reversed(range(cfg.layers)):
        x, z, qh, sh, up, down = kept[i]
        q, s, qt, st, grads[f"down_bias{i}"] = fp8bs.fp8_quant_epilogue_backward(dy, None)
        dh = fp8bs.fp8_block_gemm(q, s, down[2], down[3])
        grads[f"down{i}"] = _weight_grad(qt, st, _decode(qh, sh))
        q, s, qt, st, grads[f"up_bias{i}"] = fp8bs.fp8_quant_epilogue_backward(dh, z, cfg.act)
        dy = fp8bs.fp8_block_gemm_epilogue(q, s, up[2], up[3], residual=dy)
        grads[f"up{i}"] = _weight_grad(qt, st, x)
    grads["embedding"] = torch.zeros_like(p["embedding"]).index_add_(0, tokens, dy.float())
    return loss, grads


def _head(cfg, p, x, target, ignore_index):
    """Mean loss, and the gradients of x and of the head's weight."""
    head = p["head"].to(torch.bfloat16)
    loss, lse = fp8bs.bf16_linear_xent(x, head, target, ignore_index)
    counts = (target != ignore_index) & (target >= 0) & (target < cfg.vocab)
    count = counts.sum().clamp_min(1).float()
    dloss = torch.ones_like(loss) / count
    dx, dhead = fp8bs.bf16_linear_xent_backward(x, head, target, lse, dloss, ignore_index)
    return loss.sum() / count, dx, dhead


def _gated_loss_and_grads(cfg, p, tokens, x, target, ignore_index):
    """loss_and_grads of the pre-norm gated blocks."""
    M, bf16 = x.shape[0], torch.bfloat16

    def empty(*shape, dtype=bf16):
        return torch.empty(*shape, dtype=dtype, device=x.device)

    kept, branch = [], None  # of the block before, added by the next norm
    for i in range(cfg.layers):
        up = fp8bs.fp8_quant_w_128x128_t(p[f"up{i}"].to(bf16))
        down = fp8bs.fp8_quant_w_128x128_t(p[f"down{i}"].to(bf16))
        h, n, rstd = torch.empty_like(x), torch.empty_like(x), empty(M, dtype=torch.float32)
        q, s = fp8bs.fp8_quant_rmsnorm(x, p[f"norm{i}"], residual=branch, h=h, y=n, rstd=rstd)
        z = empty(M, 2 * cfg.inner)
        qy, sy = fp8bs.fp8_block_gemm_gated_e4m3_out(q, s, up[0], up[1], act=cfg.act, z=z)
        branch = fp8bs.fp8_block_gemm(qy, sy, down[0], down[1])
        kept.append((h, n, rstd, z, up, down))
        x = h
    h, rstd = torch.empty_like(x), empty(M, dtype=torch.float32)
    y = fp8bs.bf16_rmsnorm(x, p["norm"], residual=branch, h=h, rstd=rstd)

    grads = {}
    loss, dy, grads["head"] = _head(cfg, p, y, target, ignore_index)
    dh, grads["norm"] = fp8bs.bf16_rmsnorm_backward(dy, h, rstd, p["norm"])
    for i in reversed(range(cfg.layers)):
        h, n, rstd, z, up, down = kept[i]
        q, s, qt, st, _ = fp8bs.fp8_quant_epilogue_backward(dh, None)
        dy = fp8bs.fp8_block_gemm(q, s, down[2], down[3])
        q, s, zt, szt, yt, syt = fp8bs.fp8_quant_gated_backward(dy, z, cfg.act)
        grads[f"down{i}"] = fp8bs.fp8_block_gemm_rowscaled(qt, st, yt, syt)
        grads[f"up{i}"] = _weight_grad(zt, szt, n)
        dn = fp8bs.fp8_block_gemm(q, s, up[2], up[3])
        dh, grads[f"norm{i}"] = fp8bs.bf16_rmsnorm_backward(dn, h, rstd, p[f"norm{i}"], dh=dh)
    grads["embedding"] = torch.zeros_like(p["embedding"]).index_add_(0, tokens, dh.float())
    return loss, grads


def update(p, grads, state, lr, betas=(0.9, 0.99), eps=1e-8):
    """Adam; ``state`` is a dict that starts empty."""
    t = state["t"] = state.get("t", 0) + 1
    for k, g in grads.items():
        g = g.float()
        m, v = state.setdefault(k, (torch.zeros_like(g), torch.zeros_like(g)))
        m.lerp_(g, 1 - betas[0])
        v.lerp_(g * g, 1 - betas[1])
        p[k] -= lr * (m / (1 - betas[0] ** t)) / ((v / (1 - betas[1] ** t)).sqrt() + eps)


def batch(cfg, rows, seed, device="cuda"):
    """Tokens and their images under a fixed permutation; every eighth position
    carries no loss."""
    g = torch.Generator().manual_seed(seed)
    image = torch.randperm(cfg.vocab, generator=torch.Generator().manual_seed(1))
    tokens = torch.randint(cfg.vocab, (rows,), generator=g)
    target = image[tokens]
    target[::8] = -100
    return tokens.to(device), target.to(device)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--rows", type=int, default=2000)
    ap.add_argument("--lr", type=float, default=0.01)
    ap.add_argument("--block", choices=["mlp", "gated"], default="mlp")
    a = ap.parse_args()
    cfg = Config(block=a.block, act="gelu" if a.block == "mlp" else "silu")
    p, state = init(cfg), {}
    for step in range(a.steps):
        loss, grads = loss_and_grads(cfg, p, *batch(cfg, a.rows, step))
        update(p, grads, state, a.lr)
        if step % 10 == 0 or step == a.steps - 1:
            print(f"step {step:4d}  loss {loss.item():.4f}", flush=True)


if __name__ == "__main__":
    main()
