"""Balance loss, counts and gradient against fp64.

Counts are exact.  A token's scores: exponentials of arguments up to 64 in
magnitude whose rounding is 64 * 2^-24 = 2^-18 at most, divided by their fp32
sum: 2^-17 relative with all roundings behind.  So |loss - exact| <= 2^-17
|loss| (f and p are positive) and |gradient - exact| <= coef / (S' n) p slope
(f + d) 2^-16 and half a step of its type."""

import math

import pytest
import torch

import routed_swiglu_experts_b200 as rse
from oracle import around_oracle as ao

from gpu_util import cuda_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def workspace():
    ws = torch.empty(rse.MOE_BALANCE_WS_BYTES, dtype=torch.uint8, device="cuda")
    rse.moe_workspace_init(ws)
    return ws


def config(E, k, softmax):
    return rse.make_config(128, E, k, 128, 0, 7.0, score=rse.MOE_SCORE_SOFTMAX if softmax else rse.MOE_SCORE_SIGMOID)


def inputs(T, E, k, dtype, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(T, E, generator=g) * spread - 0.5 * torch.arange(1, E + 1).log()).to(dtype)
    return z, z.float().topk(k, dim=1).indices.to(torch.int32), g


def run(z, ids, softmax, offsets=None, mask=None, coef=0.01, up=None, grad=F32, ws=None, zd=None):
    T, E = z.shape
    S = 1 if offsets is None else len(offsets) - 1
    counts = torch.full((S, E), -5, dtype=torch.int32, device="cuda")
    tokens = torch.full((S,), -5, dtype=torch.int32, device="cuda")
    loss = torch.full((1,), -5.0, device="cuda")
    g = None if grad is None else torch.full((T, E), -5.0, dtype=grad, device="cuda")
    rse.moe_balance_loss(config(E, ids.shape[1], softmax), z.cuda() if zd is None else zd, ids.cuda(), counts, tokens, loss,
                         workspace() if ws is None else ws, grad_logits=g,
                         seq_offsets=None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda(),
                         token_mask=None if mask is None else mask.cuda(), coef=coef,
                         grad_loss=None if up is None else torch.tensor([up], device="cuda"))
    return counts, tokens, loss, g


def check(got, z, ids, softmax, offsets=None, mask=None, coef=0.01, up=1.0):
    counts, tokens, loss, g = got
    z64 = z.double().requires_grad_()
    want, c, n, f = ao.balance(z64, ids, softmax, offsets, mask, coef)
    assert torch.equal(counts.cpu(), c) and torch.equal(tokens.cpu(), n)
    value = float(want.detach())
    assert abs(float(loss) - value) <= 2.0 ** -17 * abs(value)
    if g is None:
        return
    if int(n.sum()) == 0:
        assert not bool(g.any())
        return
    want.backward()
    exact = z64.grad * up
    p = ao.balance_scores(z.double(), softmax)
    whole = max(1, int((n > 0).sum()))
    per = torch.zeros(z.shape[0], dtype=torch.float64)
    ends = [0, z.shape[0]] if offsets is None else offsets
    for s in range(len(n)):
        per[max(ends[s], 0):ends[s + 1]] = abs(coef * up) / (whole * max(1, int(n[s])))
    slope = 1.0 if softmax else torch.sigmoid(-z.double())
    size = per[:, None] * p * slope * (f + (p * f).sum(1, keepdim=True))
    dt = g.dtype
    half, least = torch.finfo(dt).eps / 2, {F32: 2.0 ** -149, BF16: 2.0 ** -133, F16: 2.0 ** -24}[dt]
    err = (g.cpu().double() - exact).abs()
    bound = size * 2.0 ** -16 + exact.abs() * half * (1 + 2.0 ** -8) + least
    assert bool((err <= bound).all()), float((err - bound).max())


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("dtype,grad", [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (7, 5, 2), (64, 8, 2), (33, 37, 6), (257, 64, 6), (100, 160, 8),
                                   (40, 257, 3), (17, 512, 16), (9, 1000, 8), (12, 1024, 4)])
def test_sizes(T, E, k, dtype, grad, softmax):
    z, ids, _ = inputs(T, E, k, dtype, T * E + k)
    up = 4096.0 if grad == F16 else None
    check(run(z, ids, softmax, grad=grad, up=up), z, ids, softmax, up=up or 1.0)


@pytest.mark.parametrize("softmax", [False, True])
def test_sequences_masks_and_tokens_outside(softmax):
    T, E, k = 600, 24, 3
    z, ids, g = inputs(T, E, k, F32, 3)
    ids[5, 1], ids[6, 0], ids[7, 2] = -1, E, 2 ** 31 - 1
    mask = torch.rand(T, generator=g) < 0.7
    mask[300:310] = False                                        # a sequence of masked tokens alone
    cases = [([3, 40, 40, 300, 310, 311, 590], mask), ([0, 600], mask), ([0, 1, 2, 3, 600], None), ([600, 600], None),
             ([0, 0, 0], None), (list(range(0, 601, 2)), mask.to(torch.uint8) * 7), ([10, 20], torch.zeros(T, dtype=torch.bool))]
    for offsets, m in cases:
        check(run(z, ids, softmax, offsets, m), z, ids, softmax, offsets, m)
    check(run(z, ids, softmax, None, mask), z, ids, softmax, None, mask)


def test_offsets_outside_the_tokens_stay_inside():
    z, ids, _ = inputs(50, 8, 2, F32, 4)
    got = run(z, ids, False, [-10, 20, 80])
    check(got, z, ids, False, [0, 20, 50])


def test_what_masked_tokens_hold_does_not_matter():
    z, ids, _ = inputs(80, 16, 2, BF16, 5)
    mask = torch.arange(80) % 4 != 1
    clean = run(z, ids, True, None, mask, grad=BF16)
    z[1::4] = torch.tensor([math.nan, math.inf, -math.inf, torch.finfo(BF16).max] * 4).to(BF16)
    ids[1::4] = -1
    dirty = run(z, ids, True, None, mask, grad=BF16)
    assert all(torch.equal(a, b) for a, b in zip(clean, dirty))
    assert not bool(clean[3][1::4].any())


def test_extreme_logits():
    T, E = 8, 12
    z, ids, _ = inputs(T, E, 2, F32, 6)
    z[0], z[1] = -200.0 + z[0], 200.0 + z[1]                      # every sigmoid below fp32's range, and at 1
    z[2, 3:] = -math.inf                                          # experts that cannot be chosen
    z[3, 0] = math.inf
    z[4] = torch.finfo(F32).min
    for softmax in (False, True):
        mask = torch.ones(T, dtype=torch.bool)
        mask[3] = not softmax                                     # (the softmax of an infinity is NaN)
        counts, tokens, loss, g = run(z, ids, softmax, None, mask)
        want, c, n, f = ao.balance(z.double(), ids, softmax, None, mask, 0.01)
        assert torch.equal(counts.cpu(), c)
        # (differences of logits near 200: their rounding in the inputs is exact, exp's argument's 2^-16)
        assert abs(float(loss) - float(want)) <= 2.0 ** -14 * float(want)
        assert bool(torch.isfinite(g).all())


def test_a_nan_logit_spoils_its_token_and_the_loss_alone():
    z, ids, _ = inputs(20, 8, 2, F32, 7)
    clean = run(z, ids, False)[3]
    z[4, 1] = math.nan
    counts, tokens, loss, g = run(z, ids, False)
    assert math.isnan(float(loss)) and bool(torch.isnan(g[4]).all())
    keep = torch.arange(20) != 4
    assert torch.equal(g[keep.cuda()], clean[keep.cuda()])


def test_strided_logits_and_gradient():
    z, ids, _ = inputs(70, 33, 4, BF16, 8)
    wide = torch.full((70, 64), float("nan"), dtype=BF16, device="cuda")
    wide[:, 7:40] = z.cuda()
    big = torch.full((70, 50), 9.0, dtype=BF16, device="cuda")
    counts, tokens = torch.empty(1, 33, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    loss = torch.empty((), device="cuda")
    rse.moe_balance_loss(config(33, 4, True), wide[:, 7:40], ids.cuda(), counts, tokens, loss, workspace(), grad_logits=big[:, 3:36],
                         coef=0.01)
    check((counts, tokens, loss, big[:, 3:36].contiguous()), z, ids, True)
    assert bool((big[:, :3] == 9).all()) and bool((big[:, 36:] == 9).all())


def test_no_tokens_without_gradient_and_coefficients():
    z, ids, _ = inputs(30, 8, 2, F32, 9)
    counts, tokens, loss, _ = run(z[:0], ids[:0], False)
    assert not bool(counts.any()) and not bool(tokens.any()) and float(loss) == 0
    counts, tokens, loss, _ = run(z[:0], ids[:0], False, [0, 0, 0])
    assert not bool(counts.any()) and not bool(tokens.any()) and float(loss) == 0
    check(run(z, ids, True, grad=None), z, ids, True)
    for coef, up in ((0.0, None), (-2.0, 3.0), (1e-3, 0.0)):
        check(run(z, ids, True, coef=coef, up=up), z, ids, True, coef=coef, up=1.0 if up is None else up)


def test_many_tokens_same_result_each_time():
    """Enough tokens for every block and several rounds of them; the loss keeps its bits."""
    T, E, k = 40000, 64, 6
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn(T, E, generator=g, device="cuda") * 1.5
    ids = z.topk(k, dim=1).indices.to(torch.int32)
    offsets = torch.tensor([0, 17000, 17001, 30000, 40000], dtype=torch.int32, device="cuda")
    cfg, ws = config(E, k, False), workspace()
    seen = []
    for _ in range(4):
        counts, tokens = torch.empty(4, E, dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")
        loss, grad = torch.empty((), device="cuda"), torch.empty(T, E, device="cuda")
        rse.moe_balance_loss(cfg, z, ids, counts, tokens, loss, ws, grad_logits=grad, seq_offsets=offsets, coef=0.01)
        seen.append((counts, tokens, loss, grad))
    for other in seen[1:]:
        assert all(torch.equal(a, b) for a, b in zip(seen[0], other))
    counts, tokens, loss, grad = seen[0]
    seq = torch.searchsorted(offsets[1:].long(), torch.arange(T, device="cuda"), right=True)
    want = torch.bincount((seq[:, None] * E + ids).view(-1), minlength=4 * E).view(4, E)
    assert torch.equal(counts.long(), want) and tokens.tolist() == [17000, 1, 12999, 10000]
    s = torch.sigmoid(z.double())
    p = s / s.sum(1, keepdim=True)
    n = tokens.double()[seq][:, None]
    f = want.double()[seq] * (E / k) / n
    d = (p * f).sum(1, keepdim=True)
    exact = float((d / n).sum()) * 0.01 / 4
    assert abs(float(loss) - exact) <= 2.0 ** -17 * exact
    ge = p * (f - d) * (1 - s) * (0.01 / 4) / n
    size = p * (f + d) * (1 - s) * (0.01 / 4) / n
    assert bool(((grad.double() - ge).abs() <= size * 2.0 ** -16 + 2.0 ** -149).all())


def test_in_a_graph_and_on_two_streams():
    z, ids, _ = inputs(500, 64, 6, F32, 10)
    zd, idd = z.cuda(), ids.cuda()
    cfg = config(64, 6, True)
    E = 64

    def outs():
        return (torch.empty(2, E, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda"),
                torch.empty((), device="cuda"), torch.empty(500, E, device="cuda"))
    off = torch.tensor([0, 200, 500], dtype=torch.int32, device="cuda")

    def call(o, ws, stream=None):
        rse.moe_balance_loss(cfg, zd, idd, o[0], o[1], o[2], ws, grad_logits=o[3], seq_offsets=off, coef=0.01, stream=stream)
    a, ws = outs(), workspace()
    call(a, ws)
    check(a, z, ids, True, [0, 200, 500])
    b = outs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(b, ws)
        call(b, ws)
    for _ in range(2):
        for t in b:
            t.fill_(3)
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    streams, wss, both = [torch.cuda.Stream() for _ in range(2)], [workspace(), workspace()], [outs(), outs()]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, w, o in zip(streams, wss, both):
            call(o, w, s)
    torch.cuda.synchronize()
    for o in both:
        assert all(torch.equal(x, y) for x, y in zip(a, o))


def exact_on_device(z, ids, softmax, offsets, mask, coef):
    """fp64 with the device's own operators, for sizes that the plain loops take too long on."""
    (T, E), k, S = z.shape, ids.shape[1], offsets.numel() - 1
    at = torch.arange(T, device="cuda")
    seq = torch.searchsorted(offsets[1:].long(), at, right=True)
    keep = mask & (at >= offsets[0]) & (at < offsets[-1])
    seq = seq.clamp(max=S - 1)
    n = torch.zeros(S, dtype=torch.int64, device="cuda").index_add(0, seq, keep.long())
    flat = (seq[:, None] * E + ids.long()).view(-1)
    counts = torch.zeros(S * E, dtype=torch.int64, device="cuda").index_add(0, flat, keep[:, None].expand(T, k).reshape(-1).long()).view(S, E)
    p = torch.softmax(z if softmax else torch.nn.functional.logsigmoid(z), dim=1)
    per = torch.where(keep, 1 / n.clamp(min=1).double()[seq], 0.0) * (coef / max(1, int((n > 0).sum())))
    f = counts.double()[seq] * (E / k) / n.clamp(min=1).double()[seq][:, None]
    d = (p * f).sum(1, keepdim=True)
    slope = 1.0 if softmax else torch.sigmoid(-z)
    return (per * d[:, 0]).sum(), counts, n, p * (f - d) * slope * per[:, None], p * (f + d) * slope * per[:, None]


@pytest.mark.parametrize("T,E,k,S,dtype,pad", [(700, 8, 2, 600, F32, 0), (5000, 24, 3, 4000, BF16, 0), (5000, 24, 3, 4000, F32, 3),
                                               (9001, 40, 4, 300, F32, 0), (20000, 33, 4, 7, BF16, 5), (16384, 256, 8, 512, F32, 0),
                                               (3000, 512, 16, 50, F16, 0), (2001, 1000, 8, 3, F32, 0), (300, 4, 1, 100000, F32, 0),
                                               (12000, 128, 8, 1, F16, 8), (30000, 256, 8, 2, BF16, 0)])
@pytest.mark.parametrize("softmax", [False, True])
def test_large_batches_in_many_and_few_sequences(T, E, k, S, dtype, pad, softmax):
    g = torch.Generator(device="cuda").manual_seed(T + S)
    wide = (torch.randn(T, E + pad, generator=g, device="cuda") * 1.5).to(dtype)
    z = wide[:, pad // 2:pad // 2 + E]
    ids = z.float().topk(k, dim=1).indices.to(torch.int32)
    cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda").sort().values
    offsets = torch.cat([torch.tensor([5], device="cuda"), cuts.clamp(5, T - 7), torch.tensor([T - 7], device="cuda")]).to(torch.int32)
    mask = torch.rand(T, generator=g, device="cuda") < 0.8
    counts = torch.full((S, E), -5, dtype=torch.int32, device="cuda")
    tokens, loss = torch.full((S,), -5, dtype=torch.int32, device="cuda"), torch.full((), -5.0, device="cuda")
    grad = torch.full((T, E), -5.0, device="cuda")
    ws = workspace()
    for _ in range(2):
        rse.moe_balance_loss(config(E, k, softmax), z, ids, counts, tokens, loss, ws, grad_logits=grad, seq_offsets=offsets,
                             token_mask=mask, coef=0.01)
        assert rse.moe_read_device_error(ws) == 0
        want, c, n, exact, size = exact_on_device(z.double(), ids, softmax, offsets, mask, 0.01)
        assert torch.equal(counts.long(), c) and torch.equal(tokens.long(), n)
        assert abs(float(loss) - float(want)) <= 2.0 ** -17 * float(want)
        near = ((grad.double() - exact).abs() <= size * 2.0 ** -16 + 2.0 ** -149).all()
        assert bool(near)
