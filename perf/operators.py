"""The cases on which the layer's routing and its 8-bit expert products are measured.

Four operators, as a serving loop of the layer calls them:
  gate      expert selection from router logits (scores, bias, groups, top-k, weights)
  quant     bf16 rows, or weights, to e4m3 codes with power-of-two scales per 128
  gemm      products of e4m3 operands with a scale per block of 128, dense or grouped by expert
  ffn       the routed experts' SwiGLU feed-forward on e4m3 weights, bf16 in and out
"""

import math

import numpy as np
import torch

own = False

F8 = torch.float8_e4m3fn
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


def listed():
    return [
        # one decoded token of the 256-expert decode layer, groups of 32 experts: all latency
        {"name": "gate_one_token", "op": "gate", "T": 1, "E": 256, "k": 8, "score": "sigmoid", "groups": 8, "top": 4,
         "group_score": "sum2", "bias": True, "renorm": True, "alpha": 2.5, "dtype": "float32"},
        # the mid layer's 4096 tokens with a softmax router whose logits stay in bf16
        {"name": "gate_softmax_bf16", "op": "gate", "T": 4096, "E": 64, "k": 6, "score": "softmax", "groups": 1, "top": 1,
         "group_score": "max", "bias": False, "renorm": True, "alpha": 1.0, "dtype": "bfloat16"},
        # a whole prompt batch of the large prefill layer, sigmoid scores, balance bias and groups
        {"name": "gate_prefill_groups", "op": "gate", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "groups": 8, "top": 4,
         "group_score": "sum2", "bias": True, "renorm": True, "alpha": 2.5, "dtype": "float32"},
        # the mid layer's tokens quantised into their routed rows (six copies of each token, expert by expert)
        {"name": "quant_routed_rows", "op": "quant", "kind": "rows", "rows": 4096, "cols": 2048, "k": 6, "dtype": "bfloat16"},
        # weights laid out once when a bf16 model is loaded: down projections of sixteen mid-layer experts, ragged blocks
        {"name": "quant_weights", "op": "quant", "kind": "weight", "groups": 16, "rows": 2048, "cols": 1408, "dtype": "bfloat16"},
        # one decoded token through one dense projection: a stream of the weights
        {"name": "gemm_one_token", "op": "gemm", "rows": 1, "groups": 1, "N": 6144, "K": 2048, "scaled": False, "out": "bfloat16", "skew": 0.0},
        # a ragged batch through one dense projection with odd sizes (K no multiple of 128), fp32 results
        {"name": "gemm_dense_odd", "op": "gemm", "rows": 1001, "groups": 1, "N": 2808, "K": 2000, "scaled": False, "out": "float32", "skew": 0.0},
        # the mid layer's gate/up product over all its experts
        {"name": "gemm_grouped_mid", "op": "gemm", "rows": 24576, "groups": 64, "N": 2816, "K": 2048, "scaled": False, "out": "bfloat16", "skew": 0.0},
        # one rank's 32 of the large layer's 256 experts, unevenly loaded, down product with the combine weights
        {"name": "gemm_grouped_skewed", "op": "gemm", "rows": 16384, "groups": 32, "N": 6144, "K": 2048, "scaled": True, "out": "bfloat16", "skew": 0.5},
        # decode: 32 tokens of the large layer on one rank's share of experts, a few rows for each
        {"name": "ffn_decode", "op": "ffn", "T": 32, "H": 6144, "I": 2048, "E": 64, "k": 8, "limit": 7.0, "skew": 0.0},
        # the mid layer's routed feed-forward
        {"name": "ffn_mid", "op": "ffn", "T": 4096, "H": 2048, "I": 1408, "E": 64, "k": 6, "limit": 7.0, "skew": 0.0},
        # a longer prompt batch on larger experts, unevenly loaded
        {"name": "ffn_large_skewed", "op": "ffn", "T": 8192, "H": 4096, "I": 2048, "E": 32, "k": 4, "limit": 7.0, "skew": 0.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "quant", "gemm", "ffn"])
    if op == "gate":
        groups = rng.choice([1, 1, 2, 4, 5, 8, 16])
        per = _log(rng, 2, 512 // groups)
        top = rng.randint(1, groups)
        E = groups * per
        return {"op": "gate", "T": _log(rng, 1, 16384 * 256 // max(E, 256)), "E": E, "k": rng.randint(1, min(16, top * per)),
                "score": rng.choice(["sigmoid", "softmax"]), "groups": groups, "top": top,
                "group_score": rng.choice(["sum2", "max"]), "bias": rng.random() < 0.6, "renorm": rng.random() < 0.6,
                "alpha": rng.choice([1.0, 2.5]), "dtype": rng.choice(sorted(DTYPES))}
    if op == "quant":
        cols = 16 * _log(rng, 4, 384)
        if rng.random() < 0.6:
            k = rng.randint(1, 8)
            rows = _log(rng, 1, max(1, min(8192, 24576 * 2048 // (cols * k))))
            return {"op": "quant", "kind": "rows", "rows": rows, "cols": cols, "k": k, "dtype": rng.choice(sorted(DTYPES))}
        rows = _log(rng, 16, 4096)
        groups = rng.randint(1, max(1, min(16, 16 * 2048 * 1408 // (rows * cols))))
        return {"op": "quant", "kind": "weight", "groups": groups, "rows": rows, "cols": cols, "dtype": rng.choice(sorted(DTYPES))}
    if op == "gemm":
        groups = rng.choice([1, 1, _log(rng, 2, 64)])
        N, K = 8 * _log(rng, 8, 768), 16 * _log(rng, 8, 384)
        groups = max(1, min(groups, 64 * 2816 * 2048 // (N * K)))
        rows = _log(rng, 1, max(1, min(16384, 16384 * 6144 * 2048 // (2 * N * K))))
        return {"op": "gemm", "rows": rows, "groups": groups, "N": N, "K": K, "scaled": rng.random() < 0.5,
                "out": rng.choice(["bfloat16", "float32"]), "skew": rng.choice([0.0, 0.5]) if groups > 1 else 0.0}
    H, I = 128 * _log(rng, 1, 32), 128 * _log(rng, 1, 16)
    E = _log(rng, 2, max(2, min(64, 32 * 4096 * 2048 // (H * I))))
    k = rng.randint(1, min(8, E))
    T = _log(rng, 1, max(1, min(8192, 8192 * 4 * 4096 * 2048 // (2 * H * I * k))))
    return {"op": "ffn", "T": T, "H": H, "I": I, "E": E, "k": k, "limit": rng.choice([0.5, 7.0, 1e30]), "skew": rng.choice([0.0, 0.5])}


# ------------------------------------------------------------- inputs -------

def _blocks(n):
    return (n + 127) // 128


def _codes(g, *shape):
    """Random e4m3 codes with the spread that quantised normal values have."""
    q = torch.empty(shape, dtype=F8, device="cuda")
    for part in q.view(-1, shape[-1]).split(1 << 16):
        part.copy_((torch.randn(part.shape, generator=g, device="cuda") * 110.0).clamp_(-448, 448))
    return q


def _offsets(rows, groups, skew, g):
    """Row offsets of the groups: every row falls to a group by itself, later groups less often when skewed."""
    p = 1.0 / torch.arange(1, groups + 1, dtype=torch.float32, device="cuda") ** (2 * skew)
    ids = torch.multinomial(p, rows, replacement=True, generator=g)
    counts = torch.bincount(ids, minlength=groups)
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


def _routed(T, E, k, skew, g):
    """Slots sorted by expert (src) and the experts' offsets, each token on k distinct experts."""
    z = torch.randn(T, E, generator=g, device="cuda") - skew * torch.arange(1, E + 1, device="cuda").log()
    ids = z.topk(k, dim=1).indices.reshape(-1)
    src = torch.sort(ids, stable=True).indices.to(torch.int32)
    counts = torch.bincount(ids, minlength=E)
    return src, torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    rand = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    s = {"case": c}
    if c["op"] == "gate":
        s["logits"] = (randn(c["T"], c["E"]) * 1.5).to(DTYPES[c["dtype"]])
        s["bias"] = rand(c["E"]) * 0.2 - 0.1 if c["bias"] else None
        s["ids"] = torch.empty(c["T"], c["k"], dtype=torch.int32, device="cuda")
        s["w"] = torch.empty(c["T"], c["k"], device="cuda")
    elif c["op"] == "quant":
        if c["kind"] == "rows":
            s["x"] = (randn(c["rows"], c["cols"]) * (0.05 + 4 * rand(c["rows"], 1))).to(DTYPES[c["dtype"]])
            s["src"] = torch.randperm(c["rows"] * c["k"], generator=g, device="cuda").to(torch.int32)
            n = c["rows"] * c["k"]
            s["q"] = torch.empty(n, c["cols"], dtype=F8, device="cuda")
            s["s"] = torch.empty(_blocks(c["cols"]), n, device="cuda")
        else:
            s["x"] = (randn(c["groups"], c["rows"], c["cols"]) / math.sqrt(c["cols"])).to(DTYPES[c["dtype"]])
            s["q"] = torch.empty(c["groups"], c["rows"], c["cols"], dtype=F8, device="cuda")
            s["s"] = torch.empty(c["groups"], _blocks(c["rows"]), _blocks(c["cols"]), device="cuda")
    elif c["op"] == "gemm":
        n, G, N, K = c["rows"], c["groups"], c["N"], c["K"]
        s["a"], s["w"] = _codes(g, n, K), _codes(g, G, N, K)
        s["sa"] = torch.exp2(torch.randint(-8, -5, (_blocks(K), n), generator=g, device="cuda").float())
        s["sw"] = (0.5 + rand(G, _blocks(N), _blocks(K))) / (110.0 * math.sqrt(K))
        s["offsets"] = _offsets(n, G, c["skew"], g) if G > 1 else None
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max()) if G > 1 else n
        s["c"] = rand(n) if c["scaled"] else None
        s["out"] = torch.empty(n, N, dtype=DTYPES[c["out"]], device="cuda")
    else:
        T, H, I, E, k = (c[n] for n in ("T", "H", "I", "E", "k"))
        s["x"] = randn(T, H).to(torch.bfloat16)
        s["w1"], s["w2"] = _codes(g, E, 2 * I, H), _codes(g, E, H, I)
        s["s1"] = (0.5 + rand(E, 2 * I // 128, H // 128)) / (110.0 * math.sqrt(H))
        s["s2"] = (0.5 + rand(E, H // 128, I // 128)) / (110.0 * math.sqrt(I))
        s["src"], s["offsets"] = _routed(T, E, k, c["skew"], g)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        s["c"] = rand(T * k)
        s["out"] = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda")
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program of the framework keeps beside its tensors: the layer's configuration, weight handles and workspace."""
    import routed_swiglu_experts_b200 as rse
    c = s["case"]
    if c["op"] == "gate":
        s["cfg"] = rse.make_config(
            128, c["E"], c["k"], 128, 0, 7.0, c["alpha"], c["renorm"],
            score=rse.MOE_SCORE_SOFTMAX if c["score"] == "softmax" else rse.MOE_SCORE_SIGMOID, num_groups=c["groups"],
            top_groups=c["top"], group_score=rse.MOE_GROUP_MAX if c["group_score"] == "max" else rse.MOE_GROUP_SUM2)
    elif c["op"] == "gemm":
        s["ws"] = torch.empty(rse.MOE_WS_HEADER_BYTES, dtype=torch.uint8, device="cuda")
        rse.moe_workspace_init(s["ws"])
    elif c["op"] == "ffn":
        s["cfg"] = rse.make_config(c["H"], c["E"], c["k"], c["I"], 0, c["limit"], expert_format=rse.MOE_W_FP8_B128)
        s["handle"] = rse.make_weights(w_gate_up=s["w1"], s_gate_up=s["s1"], w_down=s["w2"], s_down=s["s2"])
        s["ws"] = torch.empty(rse.moe_workspace_size(s["cfg"], c["T"]), dtype=torch.uint8, device="cuda")
        rse.moe_workspace_init(s["ws"])


# ---------------------------------------------------------------- run -------

def _run_own(s):
    import routed_swiglu_experts_b200 as rse
    c = s["case"]
    if c["op"] == "gate":
        rse.moe_gate_topk(s["cfg"], s["logits"], s["bias"], s["ids"], s["w"])
        return {"ids": s["ids"], "w": s["w"]}
    if c["op"] == "quant":
        if c["kind"] == "rows":
            rse.moe_fp8_quantize(s["x"], s["q"], s["s"], src=s["src"], src_div=c["k"])
        else:
            rse.moe_fp8_quantize_weight(s["x"], s["q"], s["s"])
        return {"q": s["q"], "s": s["s"]}
    if c["op"] == "gemm":
        rse.moe_fp8_gemm(s["a"], s["sa"], s["w"], s["sw"], s["offsets"], s["c"], s["out"], s["ws"])
    else:
        rse.moe_grouped_swiglu_ffn_gather(s["cfg"], s["handle"], s["x"], c["T"], s["src"], s["offsets"], s["c"], s["out"], None,
                                          s["ws"])
    return {"out": s["out"]}


def _pow2_scale(amax):
    """The smallest power of two 2^e with amax <= 448 * 2^e (1 where amax is 0)."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))


def _quant_rows(x):
    """fp32 rows [n, K] to e4m3 codes [n, K] and scales [n, K/128 blocks]."""
    n, K = x.shape
    p = torch.nn.functional.pad(x, (0, -K % 128)).view(n, -1, 128)
    sc = _pow2_scale(p.abs().amax(2))
    return (p / sc[:, :, None]).to(F8).view(n, -1)[:, :K], sc


def _wide_w(w, sw):
    """The weights that codes and block scales stand for, fp32."""
    G, N, K = w.shape
    return w.float() * sw.repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]


def _by_group(rows, offsets, most):
    """[groups, most] row numbers, and which of them are rows of the group."""
    at = offsets[:-1, None].long() + torch.arange(most, device=offsets.device)
    return at.clamp(max=rows - 1), at < offsets[1:, None]


def _group_product(a, w, offsets, most):
    """a [rows, K] fp32 against w [groups, N, K] fp32 by row offsets, as one batch of padded groups."""
    if offsets is None:
        return a @ w[0].t()
    at, used = _by_group(a.shape[0], offsets, most)
    return torch.bmm(a[at], w.transpose(1, 2))[used]


def _gate(c, logits, bias):
    z = logits.double()  # 64 bits: which of two close experts comes first is a matter of the last bits
    if c["score"] == "softmax":
        e = torch.exp(z - z.amax(1, keepdim=True))
        sc = e / e.sum(1, keepdim=True)
    else:
        sc = 1 / (1 + torch.exp(-z))
    v = sc if bias is None else sc + bias.double()
    if c["groups"] > 1:
        per = v.view(v.shape[0], c["groups"], -1)
        top = torch.sort(per, dim=2, descending=True).values
        gv = top[:, :, 0] if c["group_score"] == "max" else top[:, :, :2].sum(2)
        best = torch.sort(gv, dim=1, descending=True, stable=True).indices[:, : c["top"]]
        keep = torch.zeros_like(gv, dtype=torch.bool).scatter_(1, best, True)
        v = torch.where(keep[:, :, None], per, torch.full_like(per, -math.inf)).view_as(v)
    ids = torch.sort(v, dim=1, descending=True, stable=True).indices[:, : c["k"]]
    w = torch.gather(sc, 1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "w": (w * c["alpha"]).float()}


def run(state):
    if own:
        return _run_own(state)
    s, c = state, state["case"]
    if c["op"] == "gate":
        return _gate(c, s["logits"], s["bias"])
    if c["op"] == "quant" and c["kind"] == "rows":
        q, sc = _quant_rows(s["x"].float()[(s["src"] // c["k"]).long()])
        return {"q": q, "s": sc.t().contiguous()}
    if c["op"] == "quant":
        G, N, K = s["x"].shape
        p = torch.nn.functional.pad(s["x"].float(), (0, -K % 128, 0, -N % 128))
        p = p.view(G, _blocks(N), 128, _blocks(K), 128)
        sc = _pow2_scale(p.abs().amax((2, 4)))
        q = (p / sc[:, :, None, :, None]).to(F8).view(G, _blocks(N) * 128, -1)[:, :N, :K]
        return {"q": q, "s": sc}
    if c["op"] == "gemm":
        a = s["a"].float() * s["sa"].t().repeat_interleave(128, 1)[:, : c["K"]]
        y = _group_product(a, _wide_w(s["w"], s["sw"]), s["offsets"], s["most"])
        y = y if s["c"] is None else y * s["c"][:, None]
        return {"out": y.to(DTYPES[c["out"]])}
    q, sc = _quant_rows(s["x"].float())
    rows = (q.float() * sc.repeat_interleave(128, 1))[(s["src"] // c["k"]).long()]
    gu = _group_product(rows, _wide_w(s["w1"], s["s1"]), s["offsets"], s["most"])
    gate, up = gu[:, : c["I"]].clamp(max=c["limit"]), gu[:, c["I"]:].clamp(-c["limit"], c["limit"])
    q, sc = _quant_rows(gate / (1 + torch.exp(-gate)) * up)
    y = _group_product(q.float() * sc.repeat_interleave(128, 1), _wide_w(s["w2"], s["s2"]), s["offsets"], s["most"])
    return {"out": (y * s["c"][:, None]).to(torch.bfloat16)}


def work(case):
    c = case
    if c["op"] == "gate":
        size = 4 if c["dtype"] == "float32" else 2
        return {"bytes": c["T"] * (c["E"] * size + c["k"] * 8) + c["E"] * 4 * c["bias"], "flops": 8 * c["T"] * c["E"]}
    if c["op"] == "quant":
        size = 4 if c["dtype"] == "float32" else 2
        if c["kind"] == "rows":
            n = c["rows"] * c["k"]
            return {"bytes": c["rows"] * c["cols"] * size + n * (4 + c["cols"] + 4 * _blocks(c["cols"])), "flops": 2 * n * c["cols"]}
        n = c["groups"] * c["rows"] * c["cols"]
        return {"bytes": n * (size + 1) + 4 * c["groups"] * _blocks(c["rows"]) * _blocks(c["cols"]), "flops": 2 * n}
    if c["op"] == "gemm":
        n, N, K = c["rows"], c["N"], c["K"]
        G = min(c["groups"], n)
        size = 4 if c["out"] == "float32" else 2
        return {"bytes": n * (K + 4 * _blocks(K) + N * size + 4 * c["scaled"]) + G * (N * K + 4 * _blocks(N) * _blocks(K)),
                "flops": 2 * n * N * K}
    T, H, I, E, k = (c[n] for n in ("T", "H", "I", "E", "k"))
    touched = E * (1 - (1 - k / E) ** T)  # experts that some token goes to
    return {"bytes": T * H * 2 + T * k * (H * 2 + 8) + touched * 3 * H * I * (1 + 4 / 16384), "flops": 6 * T * k * H * I}


# -------------------------------------------------------------- exact -------

def _rne_e4m3(x):
    """fp64 values to the nearest e4m3 value (ties to even), |x| <= 448 up to rounding."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30)))
    e = torch.where(torch.exp2(e) > x.abs(), e - 1, e)
    step = torch.exp2(e.clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_quant(x):
    """fp64 [..., n] in blocks of 128 along the last dimension: (codes, scale of each value)."""
    q, wide = torch.empty_like(x), torch.empty_like(x)
    for b in range(0, x.shape[-1], 128):
        part = x[..., b:b + 128]
        amax = part.abs().amax(-1, keepdim=True)
        sc = torch.exp2(torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448)))
        sc = torch.where(amax > 448 * sc, sc * 2, torch.where(amax <= 224 * sc, sc / 2, sc))
        sc = torch.where(amax > 0, sc, torch.ones_like(sc))
        q[..., b:b + 128] = _rne_e4m3(part / sc)
        wide[..., b:b + 128] = sc
    return q, wide


def _exact_gate(c, logits, bias):
    z = logits.double().cpu().numpy()
    T, E = z.shape
    if c["score"] == "softmax":
        top = z.max(1, keepdims=True)
        sc = np.exp(z - (top + np.log(np.exp(z - top).sum(1, keepdims=True))))
    else:
        sc = np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))
    v = sc + (0 if bias is None else bias.double().cpu().numpy())
    if c["groups"] > 1:
        per = v.reshape(T, c["groups"], E // c["groups"])
        best = np.partition(per, -1, 2)[:, :, -1]
        if c["group_score"] == "sum2" and per.shape[2] > 1:
            best = np.partition(per, -2, 2)[:, :, -2:].sum(2)
        rank = np.argsort(np.argsort(-best, axis=1, kind="stable"), axis=1, kind="stable")
        v = np.where((rank < c["top"])[:, :, None], per, -np.inf).reshape(T, E)
    ids = np.argsort(-v, axis=1, kind="stable")[:, : c["k"]]
    w = np.take_along_axis(sc, ids, 1)
    w = w * (c["alpha"] / w.sum(1, keepdims=True) if c["renorm"] else c["alpha"])
    return {"ids": torch.from_numpy(ids.astype(np.int32)), "w": torch.from_numpy(w)}


def _exact_product(a, w, sw, offsets):
    """Group by group in fp64; a holds the values themselves."""
    G, N, K = w.shape
    y = torch.empty(a.shape[0], N, dtype=torch.float64, device=a.device)
    ends = offsets.tolist() if offsets is not None else [0, a.shape[0]]
    for i in range(G):
        if ends[i + 1] > ends[i]:
            rep = torch.kron(sw[i].double(), torch.ones(128, 128, dtype=torch.float64, device=a.device))[:N, :K]
            y[ends[i]:ends[i + 1]] = a[ends[i]:ends[i + 1]] @ (w[i].double() * rep).t()
    return y


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "gate":
        return _exact_gate(c, s["logits"], s["bias"])
    if c["op"] == "quant" and c["kind"] == "rows":
        q, sc = _exact_quant(s["x"].double())
        token = torch.div(s["src"], c["k"], rounding_mode="floor").long()
        return {"q": q[token], "s": sc[:, ::128].t()[:, token]}
    if c["op"] == "quant":
        G, N, K = s["x"].shape
        x = s["x"].double()
        q, sc = torch.empty_like(x), torch.empty(s["s"].shape, dtype=torch.float64, device="cuda")
        for i in range(_blocks(N)):
            for j in range(_blocks(K)):
                part = x[:, 128 * i:128 * i + 128, 128 * j:128 * j + 128]
                amax = part.abs().flatten(1).amax(1)
                e = torch.ceil(torch.log2(amax / 448))
                e = torch.where(amax > 448 * torch.exp2(e), e + 1, torch.where(amax <= 224 * torch.exp2(e), e - 1, e))
                sc[:, i, j] = torch.exp2(e)
                q[:, 128 * i:128 * i + 128, 128 * j:128 * j + 128] = _rne_e4m3(part / torch.exp2(e)[:, None, None])
        return {"q": q, "s": sc}
    if c["op"] == "gemm":
        a = s["a"].double() * torch.kron(s["sa"].t().contiguous().double(), torch.ones(1, 128, dtype=torch.float64, device="cuda"))[:, : c["K"]]
        y = _exact_product(a, s["w"], s["sw"], s["offsets"])
        return {"out": y if s["c"] is None else y * s["c"].double()[:, None]}
    q, sc = _exact_quant(s["x"].double())
    rows = (q * sc)[torch.div(s["src"], c["k"], rounding_mode="floor").long()]
    gu = _exact_product(rows, s["w1"], s["s1"], s["offsets"])
    gate, up = torch.clamp(gu[:, : c["I"]], max=c["limit"]), torch.clamp(gu[:, c["I"]:], -c["limit"], c["limit"])
    q, sc = _exact_quant(gate * torch.sigmoid(gate) * up)
    return {"out": _exact_product(q * sc, s["w2"], s["s2"], s["offsets"]) * s["c"].double()[:, None]}
