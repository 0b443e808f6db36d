"""Quantisation-aware training on top of the library.

"BCJR-QAT: A Differentiable Relaxation of Trellis-Coded Weight Quantization"
(Technical Summary, "Core Mechanism" and "Key Technical Innovations"): the soft
codeword of the latent weights w stands in for the quantised weights, T is
annealed from T0 towards a near-zero T_end, and the schedule that skips the
high-T phase (T0 = 0.3 instead of 1.0) avoids drifting into a worse Voronoi
basin.  The drift-budget criterion compares the cumulative drift
eta * N * g_max with the basin radius (about 1e-3).

By self-reconstruction with plain gradient descent, each step is one
``bcjr_qat_step`` call (soft codeword, loss sum ||w_hat - w*||^2 and its upstream
gradient, VJP and the in-place update, all in the library's kernels); this module
only schedules T and reports.

With activations X of the layer the loss is that of its outputs ("Experimental
Results": per-layer reconstruction MSE), ||X (w_hat - w*)^T||^2 / tokens, its
products and those of its gradient on 8-bit operands (``layer_loss``; ``products``
says which, or asks for fp32).  With ``optimizer="muon"`` the latent weights are updated as one matrix by
``bcjr_muon_step``.

    python -m bcjr_sum_product_b200.qat --workload qtip --seqs 256 --T0 0.3 --T-end 0.01 --steps 40 --lr 1e-3
    python -m bcjr_sum_product_b200.qat --seqs 1024 --loss layer --tokens 512 --optimizer muon --lr 1e-2
"""
from __future__ import annotations

import argparse
import json
import math
from typing import Dict, List, Optional, Tuple

import torch

from . import lib


def anneal(T0: float, T_end: float, steps: int) -> List[float]:
    """Geometric schedule from T0 to T_end over `steps` steps (T0 only for one step)."""
    if not (T0 > 0 and T_end > 0 and steps >= 1):
        raise ValueError("T0, T_end > 0 and steps >= 1 required")
    if steps == 1:
        return [float(T0)]
    r = (T_end / T0) ** (1.0 / (steps - 1))
    return [float(T0 * r ** i) for i in range(steps)]


def hard_mse(states: torch.Tensor, codebook: torch.Tensor, target: torch.Tensor, V: int) -> torch.Tensor:
    """Per-sequence sum of squared differences between the codewords of a
    state path and the target weights (host-side report, not the hot path)."""
    cw = codebook.reshape(codebook.shape[0], -1)[states.long()]          # [n_seq, n, V]
    return ((cw.reshape(target.shape) - target) ** 2).sum(dim=1)


def layer_operands(x: torch.Tensor, stream=None) -> Tuple[torch.Tensor, ...]:
    """8-bit codes and scales of a layer's activations [tokens, in], along both axes:
    what layer_loss takes, made once for a batch of tokens."""
    return lib.fp8_quantise(x, layout="both", stream=stream)


#: How the products of a layer's loss and gradient run: on 8-bit operands, with R's codes in e5m2 or e4m3, or in fp32.
PRODUCTS = ("e5m2", "e4m3", "fp32")


def layer_loss(soft: torch.Tensor, w_target: torch.Tensor, operands: Tuple[torch.Tensor, ...], stream=None,
               r_dtype: torch.dtype = torch.float8_e5m2) -> Tuple[torch.Tensor, torch.Tensor]:
    """Change of a layer's outputs, R = X (soft - w_target)^T, [tokens, out] in bf16, and
    the gradient 2 R^T X / tokens of ||R||^2 / tokens with respect to soft, [out, in] in
    fp32.  soft and w_target are [out, in]; the residual is quantised in 128 x 128
    blocks of e4m3, R down its columns in ``r_dtype``: e5m2, or e4m3 with one more bit.
    512 normal activations on a 2048 x 2048 layer, against fp32 (layer_loss_fp32) in the
    2-norm: R is off by 3.7 %, the gradient by 6.4 % with e5m2 and by 4.9 % with e4m3."""
    x, sx, xt, sxt = operands
    tokens = x.shape[0]
    d, sd = lib.fp8_quantise(soft, 128, minus=w_target, stream=stream)
    r = lib.fp8_matmul(x, sx, d, sd, stream=stream)
    rt, srt = lib.fp8_quantise(r, 1, r_dtype, layout="cols", stream=stream)
    g = lib.fp8_matmul(rt, srt, xt, sxt, alpha=2.0 / tokens, out_dtype=torch.float32, stream=stream)
    return r, g


def layer_loss_fp32(soft: torch.Tensor, w_target: torch.Tensor, x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """layer_loss in fp32 throughout, of the activations themselves: for a driver that wants
    the gradient exactly rather than fast."""
    x = x.float()
    r = x @ (soft - w_target).t()
    return r, (2.0 / x.shape[0]) * (r.t() @ x)


def run(w_target: torch.Tensor, codebook: torch.Tensor, L: int, k: int, V: int, T0: float, T_end: float,
        steps: int, lr_w: float, lr_c: float = 0.0, stream=None, x: Optional[torch.Tensor] = None,
        shape: Optional[Tuple[int, int]] = None, optimizer: str = "sgd", mu: float = 0.95,
        weight_decay: float = 0.0, products: str = "e5m2") -> Dict:
    """Anneal from w = w_target; returns the loss history, the drift budget and
    how far the hard (Viterbi) code moved from the PTQ code of w_target.

    With ``x`` ([tokens, in]) the loss is the layer's (layer_loss, with R's codes in
    ``products`` e5m2 or e4m3, or layer_loss_fp32) and the
    sequences are the rows of a matrix of ``shape`` (out, in), cut one after the
    other; ``optimizer`` "muon" updates that matrix by lib.muon_step with momentum
    ``mu`` and ``weight_decay`` (the codebook by plain gradient descent, at lr_c)."""
    if optimizer not in ("sgd", "muon"):
        raise ValueError('optimizer must be "sgd" or "muon"')
    if products not in PRODUCTS:
        raise ValueError('products must be "e5m2", "e4m3" or "fp32"')
    by_matrix = x is not None or optimizer == "muon"
    if by_matrix:
        if shape is None or shape[0] * shape[1] != w_target.numel():
            raise ValueError("shape (out, in) must have as many entries as w_target")
        if x is not None and (x.dim() != 2 or x.shape[0] < 1 or x.shape[1] != shape[1]):
            raise ValueError("x must be [tokens, in]")
    elif weight_decay != 0.0:
        raise ValueError("weight_decay needs a layer loss or the muon optimizer")
    if stream is not None:
        # everything of the run, allocations included, on that stream, after the caller's and before its next
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=w_target.device)
        caller = torch.cuda.current_stream(w_target.device)
        stream.wait_stream(caller)
        with torch.cuda.stream(stream):
            out = run(w_target, codebook, L, k, V, T0, T_end, steps, lr_w, lr_c, None, x, shape, optimizer, mu, weight_decay,
                      products)
        caller.wait_stream(stream)
        for t in (out["w"], out["codebook"]):
            t.record_stream(caller)
        return out
    w = w_target.clone()
    c = codebook.clone()
    temps = anneal(T0, T_end, steps)
    loss_hist, gmax_hist = [], []
    soft = torch.empty_like(w)
    loss = torch.empty(w.shape[0], device=w.device)
    gw = torch.empty_like(w)
    gc = torch.empty_like(c)
    if by_matrix:
        operands = layer_operands(x) if x is not None and products != "fp32" else None
        r_dtype = torch.float8_e4m3fn if products == "e4m3" else torch.float8_e5m2
        logZ = torch.empty(w.shape[0], device=w.device)
        momentum = torch.zeros_like(w) if optimizer == "muon" else None
    for T in temps:
        if not by_matrix:
            lib.qat_step(w, w_target, c, L, k, V, T, lr_w, lr_c, out_soft=soft, out_loss=loss, grad_w=gw,
                         grad_codebook=gc)
            loss_hist.append(float(loss.sum()))
        else:
            lib.soft_codeword(w, c, L, k, V, T, out_soft=soft, out_logZ=logZ)
            if x is not None:
                pair = soft.view(shape), w_target.view(shape)
                r, g = layer_loss_fp32(*pair, x) if operands is None else layer_loss(*pair, operands, r_dtype=r_dtype)
                loss_hist.append(float(r.float().square().sum()) / x.shape[0])
            else:
                g = 2.0 * (soft - w_target)
                loss_hist.append(float(g.square().sum()) / 4.0)
            lib.vjp(w, c, L, k, V, T, g.view(w.shape), grad_w=gw, grad_codebook=gc)
            if optimizer == "muon":
                lib.muon_step(w.view(shape), gw.view(shape), momentum.view(shape), lr_w, mu=mu, weight_decay=weight_decay)
            else:
                w.mul_(1.0 - lr_w * weight_decay).sub_(gw, alpha=lr_w)
            if lr_c != 0.0:
                c.sub_(gc, alpha=lr_c)
        gmax_hist.append(float(gw.abs().max()))
    ptq_states, ptq_cost = lib.viterbi_decode(w_target, codebook, L, k, V)
    new_states, _ = lib.viterbi_decode(w, c, L, k, V)
    mse_ptq = hard_mse(ptq_states, codebook, w_target, V)
    mse_new = hard_mse(new_states, c, w_target, V)
    changed = (new_states != ptq_states).float().mean().item()
    drift = float((w - w_target).abs().max())
    # a step moves an entry by lr |gradient|, or with Muon by lr scale |orthogonalised update| (at most about 1.2), and
    # by its decay
    g_step = max(gmax_hist) if optimizer == "sgd" else 1.2 * math.sqrt(max(1.0, shape[0] / shape[1]))
    budget = lr_w * steps * (g_step + weight_decay * float(w_target.abs().max()))
    out = {}
    if x is not None:
        out.update(_layer_report(ptq_states, codebook, new_states, c, w_target, x, shape))
    return {**out, "temps": [temps[0], temps[-1]], "steps": steps, "lr_w": lr_w, "lr_c": lr_c,
            "loss_first": loss_hist[0], "loss_last": loss_hist[-1], "loss": loss_hist,
            "drift_budget": budget, "max_drift": drift, "g_max": max(gmax_hist),
            "code_changed_fraction": changed,
            "hard_mse_ptq": float(mse_ptq.sum()), "hard_mse_qat": float(mse_new.sum()),
            "w": w, "codebook": c}


def _layer_report(ptq_states, ptq_codebook, new_states, codebook, w_target, x, shape) -> Dict:
    """Change of the layer's outputs per token with the two hard codes (fp32, a report)."""
    def error(states, c):
        d = c.reshape(c.shape[0], -1)[states.long()].reshape(shape) - w_target.view(shape)
        return float((x.float() @ d.t()).square().sum()) / x.shape[0]
    return {"hard_layer_mse_ptq": error(ptq_states, ptq_codebook), "hard_layer_mse_qat": error(new_states, codebook)}


def main(argv: Optional[List[str]] = None) -> int:
    from . import inputs as I
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--workload", default="qtip", choices=sorted(I.WORKLOADS))
    ap.add_argument("--seqs", type=int, default=256)
    ap.add_argument("--T0", type=float, default=0.3)
    ap.add_argument("--T-end", type=float, default=0.01)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--lr", type=float, default=1e-3)
    ap.add_argument("--lr-c", type=float, default=0.0)
    ap.add_argument("--loss", choices=("weights", "layer"), default="weights",
                    help="reconstruct the weights, or the layer's outputs on synthetic N(0, 1) activations")
    ap.add_argument("--tokens", type=int, default=512, help="activations of --loss layer")
    ap.add_argument("--products", choices=PRODUCTS, default="e5m2",
                    help="products of --loss layer: 8-bit operands (the outputs' change in e5m2 or e4m3), or fp32")
    ap.add_argument("--optimizer", choices=("sgd", "muon"), default="sgd")
    ap.add_argument("--mu", type=float, default=0.95, help="momentum of --optimizer muon")
    ap.add_argument("--weight-decay", type=float, default=0.0)
    a = ap.parse_args(argv)
    wl = I.WORKLOADS[a.workload]
    shape = None
    if a.loss == "layer" or a.optimizer == "muon":
        # whole rows of the workload's first matrix
        n, cols = min(a.seqs, wl.n_seq) * wl.seq_len, wl.matrices[0][1]
        if n < 1 or n % cols or n > wl.matrices[0][0] * cols:
            ap.error(f"--seqs must make whole rows of {cols} weights of the first matrix (1 to {wl.matrices[0][0]} rows)")
        if a.tokens < 1:
            ap.error("--tokens must be positive")
        shape = (n // cols, cols)
    elif a.weight_decay != 0.0:
        ap.error("--weight-decay needs --loss layer or --optimizer muon")
    inp = I.make(a.workload, rows=list(range(min(a.seqs, wl.n_seq))), with_grad=False)
    lib.load()
    dev = torch.device("cuda")
    x = None
    if a.loss == "layer":
        x = torch.randn((a.tokens, shape[1]), generator=torch.Generator().manual_seed(I.ACTIVATION_SEED)).to(dev)
    out = run(inp.w.to(dev), inp.c.to(dev), wl.L, wl.k, wl.V, a.T0, a.T_end, a.steps, a.lr, a.lr_c, x=x, shape=shape,
              optimizer=a.optimizer, mu=a.mu, weight_decay=a.weight_decay, products=a.products)
    rep = {k: v for k, v in out.items() if k not in ("w", "codebook", "loss")}
    rep["loss_every_10"] = out["loss"][::10]
    rep["workload"] = a.workload
    rep["sequences"] = int(inp.w.shape[0])
    print(json.dumps(rep))
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
