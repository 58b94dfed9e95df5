"""CPU oracle (fp64) of expert selection from logits and of the block-scaled
FP8 products.  TEST INFRASTRUCTURE, as ``moe_oracle``: it shares no code with
the CUDA path.

Selection: scores sigmoid or softmax; the bias steers selection only; a
group's value is the sum of its two largest biased scores, or the largest;
ties go to the lower group and the lower id.  Token by token, in Python.

FP8: E4M3 codes are chosen by distance from the table of the format's values
(``moe_oracle.e4m3_value``), ties to the even code; a block of 128 has the
smallest power-of-two scale that brings its largest value to 448 or below.
"""

from __future__ import annotations

import math

import torch

from .moe_oracle import _cpu64, e4m3_value, f64, swiglu_clamped


def gate_scores(row, softmax: bool):
    """fp64 scores of one token's logits (a list of floats)."""
    if not softmax:
        return [1.0 / (1.0 + math.exp(-l)) if l > -700 else 0.0 for l in row]
    top = max(row)
    if top == -math.inf:
        return [0.0] * len(row)
    e = [math.exp(l - top) for l in row]
    z = math.fsum(e)
    return [x / z for x in e]


def gate_select(logits, bias, k, alpha=1.0, renorm=False, softmax=False, groups=1, top_groups=1, group_max=False):
    """(ids int64 [T, k], weights fp64 [T, k]).  Without a bias equal scores
    of different logits keep the order of the logits."""
    ids, weights = [], []
    b = None if bias is None else _cpu64(bias).tolist()
    for row in _cpu64(logits).tolist():
        E = len(row)
        s = gate_scores(row, softmax)
        v = s if b is None else [x + y for x, y in zip(s, b)]
        order = row if b is None else v
        allowed = range(E)
        if groups > 1:
            per = E // groups
            val = []
            for g in range(groups):
                part = sorted(v[g * per:(g + 1) * per], reverse=True)
                raw = sorted(order[g * per:(g + 1) * per], reverse=True)
                val.append(raw[0] if group_max else sum(part[:2]))
            kept = sorted(range(groups), key=lambda g: (-val[g], g))[:top_groups]
            allowed = [e for g in sorted(kept) for e in range(g * per, (g + 1) * per)]
        chosen = sorted(allowed, key=lambda e: (-order[e], e))[:k]
        w = [s[e] for e in chosen]
        total = math.fsum(w)
        if renorm:
            w = [x / total if total else 0.0 for x in w]
        ids.append(chosen)
        weights.append([alpha * x for x in w])
    return torch.tensor(ids, dtype=torch.int64).reshape(-1, k), torch.tensor(weights, dtype=f64).reshape(-1, k)


_CODES = e4m3_value(torch.arange(127, dtype=torch.int64).to(torch.uint8))  # 0, the positive values, ascending
_MID = (_CODES[1:] + _CODES[:-1]) / 2


def e4m3_nearest(x: torch.Tensor) -> torch.Tensor:
    """The E4M3 value nearest to each fp64 value (ties to the even code,
    magnitudes above 448 to 448)."""
    mag = x.abs()
    up = torch.searchsorted(_MID, mag, right=True)     # a value on a border goes up ...
    lo = torch.searchsorted(_MID, mag, right=False)
    code = torch.where((up != lo) & (up % 2 == 1), lo, up)  # ... unless the code above is odd
    return torch.sign(x) * _CODES[code]


def block_scale(amax: float) -> float:
    if amax == 0:
        return 1.0
    e = -126
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def quantize_rows(x: torch.Tensor):
    """fp64 rows [n, K] -> (code values [n, K], scales [ceil(K/128), n])."""
    x = _cpu64(x)
    n, K = x.shape
    q, s = torch.empty_like(x), torch.empty((K + 127) // 128, n, dtype=f64)
    for r in range(n):
        for b in range(s.shape[0]):
            part = x[r, 128 * b:128 * b + 128]
            s[b, r] = block_scale(float(part.abs().max()))
            q[r, 128 * b:128 * b + 128] = e4m3_nearest(part / s[b, r])
    return q, s


def quantize_weight(w: torch.Tensor):
    """[G, N, K] -> (code values, scales [G, ceil(N/128), ceil(K/128)])."""
    w = _cpu64(w)
    G, N, K = w.shape
    q, s = torch.empty_like(w), torch.empty(G, (N + 127) // 128, (K + 127) // 128, dtype=f64)
    for g in range(G):
        for i in range(s.shape[1]):
            for j in range(s.shape[2]):
                at = (g, slice(128 * i, 128 * i + 128), slice(128 * j, 128 * j + 128))
                s[g, i, j] = block_scale(float(w[at].abs().max()))
                q[at] = e4m3_nearest(w[at] / s[g, i, j])
    return q, s


def wide_rows(q: torch.Tensor, s: torch.Tensor) -> torch.Tensor:
    """The values codes [n, K] and scales [blocks, n] stand for."""
    return q * s.T.repeat_interleave(128, dim=1)[:, : q.shape[1]]


def wide_weight(q: torch.Tensor, s: torch.Tensor) -> torch.Tensor:
    G, N, K = q.shape
    return q * s.repeat_interleave(128, dim=1)[:, :N].repeat_interleave(128, dim=2)[:, :, :K]


def gemm(a, sa, w, sw, offsets=None, row_scale=None):
    """(out fp64 [rows, N], sum of the terms' magnitudes); rows of no group are NaN."""
    A, W = wide_rows(_cpu64(a), _cpu64(sa)), wide_weight(_cpu64(w), _cpu64(sw))
    rows = A.shape[0]
    ends = [0, rows] if offsets is None else [int(v) for v in offsets]
    out = torch.full((rows, W.shape[1]), math.nan, dtype=f64)
    mag = torch.zeros_like(out)
    for g in range(W.shape[0]):
        r0, r1 = ends[g], ends[g + 1]
        c = 1.0 if row_scale is None else _cpu64(row_scale)[r0:r1, None]
        out[r0:r1] = (A[r0:r1] @ W[g].T) * c
        mag[r0:r1] = (A[r0:r1].abs() @ W[g].abs().T) * (c if row_scale is None else c.abs())
    return out, mag


def ffn(x_rows, w1, s1, w2, s2, offsets, limit, row_scale=None):
    """Routed rows x_rows [R, H] through FP8 experts: rows and activations quantised."""
    I = w2.shape[2]
    q, s = quantize_rows(x_rows)
    gu, _ = gemm(q, s, w1, s1, offsets)
    h, hs = quantize_rows(swiglu_clamped(gu[:, :I], gu[:, I:], limit))
    return gemm(h, hs, w2, s2, offsets, row_scale)[0]
