"""fp64 forms of the operators around the routed layer: RMS norm with 8-bit
rows, request adapters, balance loss.  Plain loops over rows and sequences;
inputs are CPU tensors."""

from __future__ import annotations

import math

import torch

from .gate_fp8_oracle import quantize_rows


def rmsnorm(x, weight, eps, residual=None):
    """(h, y): the sum in the residual's type (x's own values without one), and
    the normalised rows in fp64."""
    h = x if residual is None else (x.float() + residual.float()).to(residual.dtype)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    rows = []
    for r in h.double():
        rows.append(r / math.sqrt(float((r * r).sum()) / r.numel() + eps))
    y = torch.stack(rows) if rows else h.double()
    return h, y if weight is None else y * weight.double()


def norm_scales(y):
    """Scales [ceil(H/128), rows] of fp64 rows: the quantisation's."""
    return quantize_rows(y)[1]


def lora(x, a, b, scale, adapters, base):
    """(out, size): out in fp64, and the sum of its products' magnitudes."""
    T, N = x.shape[0], b.shape[1]
    out = torch.zeros(T, N, dtype=torch.float64) if base is None else base.double().clone()
    size = out.abs()
    for t in range(T):
        i = int(adapters[t])
        if 0 <= i < a.shape[0]:
            c = 1.0 if scale is None else float(scale[i])
            out[t] += c * (b[i].double() @ (a[i].double() @ x[t].double()))
            size[t] += abs(c) * (b[i].double().abs() @ (a[i].double().abs() @ x[t].double().abs()))
    return out, size


def balance_scores(z, softmax):
    """p of fp64 logits (differentiable)."""
    logs = z if softmax else torch.nn.functional.logsigmoid(z)
    return torch.softmax(logs, dim=1)


def balance(z, ids, softmax, offsets=None, mask=None, coef=1.0):
    """(loss, counts, tokens, f per token): the loss in fp64 as a function of the
    logits z (fp64, may require a gradient); f [T, E], 0 for tokens not counted."""
    T, E = z.shape
    k = ids.shape[1]
    offsets = [0, T] if offsets is None else [int(v) for v in offsets]
    S = len(offsets) - 1
    counts = torch.zeros(S, E, dtype=torch.int32)
    tokens = torch.zeros(S, dtype=torch.int32)
    rows = []
    for s in range(S):
        mine = [t for t in range(max(offsets[s], 0), min(offsets[s + 1], T)) if mask is None or bool(mask[t])]
        rows.append(mine)
        tokens[s] = len(mine)
        for t in mine:
            for e in ids[t].tolist():
                if 0 <= e < E:
                    counts[s, e] += 1
    whole = max(1, int((tokens > 0).sum()))
    loss = torch.zeros((), dtype=torch.float64)
    f = torch.zeros(T, E, dtype=torch.float64)
    for s in range(S):
        if rows[s]:
            fs = counts[s].double() * (E / (k * len(rows[s])))
            f[rows[s]] = fs
            loss = loss + (balance_scores(z[rows[s]], softmax).mean(0) * fs).sum()
    return loss * (coef / whole), counts, tokens, f
