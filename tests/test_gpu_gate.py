"""moe_gate and moe_dispatch on the GPU: against the definition in 64 bits (numpy), exact ties, switched-off
experts, NaN and infinities, strides; the layer run through a gate equals the layer with its own router."""
import numpy as np
import pytest
import torch

import quantized_grouped_gemm_gb300 as moe
from gpu_helpers import DeviceLayer, assert_output_close, to_dev, y_to_f64
from moe_workload import configs
import oracle

pytestmark = pytest.mark.gpu

F32_MAX = float(np.finfo(np.float32).max)
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# fp32 scores: the argument of the exponential is off by at most 2^-24 (|l| + |m|) with |l| <= 32 here,
# the exponential and the quotients by a few 2^-23, the sum of E terms by log2(E) 2^-24
W_RTOL = 2.0 ** -23 * (32 + 16)
# choice values nearer than this (relative to their scores) may be ranked either way; a sigmoid's argument is
# exact, so only the exponential, a sum, a quotient and the bias' sum round: four times 2^-23
GAP = {"softmax": 2 * W_RTOL, "sigmoid": 2 * 4 * 2.0 ** -23}


def reference(l, bias, E, k, score, groups, group_topk, group_score, renormalise, scale):
    """(idx, w, clear) in 64 bits; clear: no comparison that the choice rests on is within GAP, bar exact ties."""
    T = l.shape[0]
    l = l.astype(np.float64).copy()
    l[np.isnan(l)] = -np.inf
    l[l == np.inf] = F32_MAX
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            m = l.max(1, keepdims=True)
            e = np.exp(l - np.where(np.isfinite(m), m, 0.0))
            z = e.sum(1, keepdims=True)
            s = e / np.where(z > 0, z, 1.0)
    v = s if bias is None else s + bias.astype(np.float64)
    size = s + (0.0 if bias is None else np.abs(bias.astype(np.float64)))
    clear = np.ones(T, bool)

    def sorted_clear(values, sizes, upto):
        o = np.argsort(-values, 1, kind="stable")
        sv, sz = np.take_along_axis(values, o, 1), np.take_along_axis(sizes, o, 1)
        with np.errstate(invalid="ignore"):
            gap = sv[:, :-1] - sv[:, 1:]
        fine = (sv[:, :-1] == sv[:, 1:]) | (gap > GAP[score] * (sz[:, :-1] + sz[:, 1:]))
        return o, fine[:, upto]

    if groups > 1:
        b = v.reshape(T, groups, E // groups)
        best = -np.sort(-b, 2)
        worth = best[:, :, 0] if group_score == "max" else best[:, :, 0] + best[:, :, 1]
        gsize = np.broadcast_to(size.max(1, keepdims=True), worth.shape)
        o, fine = sorted_clear(worth, gsize, slice(group_topk - 1, group_topk))
        clear &= fine.all(1)
        keep = np.zeros((T, groups), bool)
        np.put_along_axis(keep, o[:, :group_topk], True, 1)
        v = np.where(np.repeat(keep, E // groups, 1), v, -np.inf)
        size = np.where(np.repeat(keep, E // groups, 1), size, 0.0)
        # a kept expert at -inf (a NaN choice value) still precedes every dropped one
        v = np.where(np.repeat(keep, E // groups, 1) & (v == -np.inf), -1e300, v)
    o, fine = sorted_clear(v, size, slice(0, k))
    clear &= fine.all(1)
    idx = o[:, :k]
    w = np.take_along_axis(s, idx, 1)
    if renormalise:
        z = w.sum(1, keepdims=True)
        w = np.where(z > 0, w / np.where(z > 0, z, 1.0), 0.0)
    return idx.astype(np.int32), w * scale, clear


def run_gate(logits, bias, T, E, k, stride=0, **kw):
    idx = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -7.0, dtype=torch.float32, device="cuda")
    cfg = moe.gate_config(T, E, k, dtype=logits.dtype, logits_stride=stride, **kw)
    moe.moe_gate(cfg, logits, bias, idx, w)
    torch.cuda.synchronize()
    assert (idx[T:] == -7).all() and (w[T:] == -7).all(), "written past the last token"
    return idx[:T].cpu().numpy(), w[:T].cpu().numpy()


CASES = [
    # T, E, k, dtype, score, groups, group_topk, group_score, bias, renormalise, scale, pad, switched off
    (1, 256, 8, "f32", "sigmoid", 8, 4, "top2", True, True, 2.5, 0, 0.0),
    (37, 256, 8, "f32", "softmax", 1, 1, "top2", False, True, 1.0, 0, 0.0),
    (1000, 256, 8, "bf16", "sigmoid", 8, 3, "max", True, False, 1.0, 8, 0.1),
    (129, 60, 6, "f16", "softmax", 1, 1, "top2", False, False, 1.0, 4, 0.2),
    (65, 512, 10, "bf16", "softmax", 16, 4, "top2", True, True, 1.0, 0, 0.0),
    (31, 1024, 32, "f32", "sigmoid", 32, 16, "max", False, True, 1.0, 1, 0.0),
    (70, 1000, 17, "f16", "softmax", 4, 2, "top2", True, True, 0.5, 3, 0.3),
    (9, 1, 1, "f32", "softmax", 1, 1, "top2", False, True, 1.0, 0, 0.0),
    (9, 3, 3, "f32", "sigmoid", 1, 1, "top2", True, True, 1.0, 0, 0.5),
    (40, 32, 32, "bf16", "softmax", 1, 1, "top2", False, True, 1.0, 0, 0.5),
    (257, 33, 5, "f32", "softmax", 11, 3, "top2", True, False, 1.0, 0, 0.0),
    (257, 96, 4, "f32", "sigmoid", 2, 1, "top2", True, True, 1.0, 0, 0.9),
    (64, 300, 1, "bf16", "softmax", 1, 1, "top2", False, True, 1.0, 4, 0.0),
    (64, 128, 2, "f16", "sigmoid", 4, 4, "top2", True, False, 1.0, 0, 0.0),
]


@pytest.mark.parametrize("T,E,k,dt,score,groups,gk,gs,with_bias,ren,scale,pad,off", CASES)
def test_gate_against_64_bits(T, E, k, dt, score, groups, gk, gs, with_bias, ren, scale, pad, off):
    g = torch.Generator().manual_seed(T * 1000 + E + k)
    l = 2.0 * torch.randn(T, E, generator=g)
    l[torch.rand(T, E, generator=g) < off] = -np.inf
    if off:
        l[:: 7] = -np.inf          # tokens with nothing left
    buf = torch.full((T, E + pad), float("nan"), dtype=DT[dt])
    buf[:, :E] = l.to(DT[dt])
    bias = 0.3 * torch.randn(E, generator=g) if with_bias else None
    idx, w = run_gate(buf.cuda(), None if bias is None else bias.cuda(), T, E, k, stride=E + pad, score=score,
                      groups=groups, group_topk=gk, group_score=gs, renormalise=ren, scale=scale)
    ri, rw, clear = reference(buf[:, :E].float().numpy(), None if bias is None else bias.numpy(), E, k, score, groups,
                              gk, gs, ren, scale)
    assert clear.mean() > 0.5 or T < 10
    assert np.array_equal(idx[clear], ri[clear])
    assert (np.abs(w - rw)[clear] <= W_RTOL * np.abs(rw)[clear] + 1e-30).all()
    for t in range(T):
        assert len(set(idx[t])) == k and idx[t].min() >= 0 and idx[t].max() < E


def test_gate_ties_go_to_the_lower_index():
    # four logit values only: nearly every comparison is an exact tie
    g = torch.Generator().manual_seed(5)
    for E, k, groups, gk in ((256, 8, 1, 1), (256, 8, 8, 4), (100, 20, 4, 2), (1024, 32, 1, 1)):
        l = torch.randint(0, 4, (200, E), generator=g).float()
        idx, w = run_gate(l.cuda(), None, 200, E, k, score="sigmoid", groups=groups, group_topk=gk)
        ri, rw, clear = reference(l.numpy(), None, E, k, "sigmoid", groups, gk, "top2", True, 1.0)
        assert clear.all() and np.array_equal(idx, ri)
        assert (np.abs(w - rw) <= W_RTOL * rw).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_nan_and_infinities(score):
    E, k = 64, 4
    l = torch.linspace(-3, 3, E).repeat(7, 1)
    l[0, 10] = float("nan")               # as if switched off
    l[1, 10] = float("inf")               # first; the two of row 2 share
    l[2, [5, 50]] = float("inf")
    l[3] = float("nan")
    l[4] = -float("inf")
    l[5] = -float("inf")
    l[5, 33] = 1.0                        # one expert left
    l[6] = -3.0e38
    ri, rw, _ = reference(l.numpy(), None, E, k, score, 1, 1, "top2", True, 1.0)
    for t in (torch.float32, torch.bfloat16):
        idx, w = run_gate(l.to(t).cuda(), None, 7, E, k, score=score)
        assert idx[1][0] == 10 and set(idx[2][:2]) == {5, 50}
        assert list(idx[3]) == [0, 1, 2, 3] == list(idx[4]) and (w[3:5] == 0).all()
        assert idx[5][0] == 33 and list(idx[5][1:]) == [0, 1, 2] and list(w[5]) == [1, 0, 0, 0]
        assert np.isfinite(w).all()
        if t == torch.float32:
            assert np.array_equal(idx[[0, 1, 2, 3, 4, 5]], ri[[0, 1, 2, 3, 4, 5]])
            assert np.abs(w[:6] - rw[:6]).max() <= W_RTOL
            if score == "softmax":
                assert np.abs(w[6] - 0.25).max() <= W_RTOL


@pytest.mark.parametrize("rest", [-86.0, -86.9])
@pytest.mark.parametrize("ones", [1, 200])
def test_gate_renormalises_the_smallest_scores(rest, ones):
    """A bias that makes experts of scores near 2^-126 the chosen ones: their weights are scale / k each, as the
    scores are equal, or 0 where the scores sum to less than 2^-126 (so count as 0), never infinite or NaN."""
    E, k, scale = 256, 8, 300.0
    logits = torch.full((1, E), rest, device="cuda")
    logits[0, :ones] = 0.0
    bias = torch.zeros(E, device="cuda")
    bias[E - k:] = torch.arange(1, k + 1, device="cuda", dtype=torch.float32) * 4
    idx, w = run_gate(logits, bias, 1, E, k, score="softmax", scale=scale)
    assert idx[0].tolist() == list(range(E - 1, E - k - 1, -1))
    total = k * np.exp(np.float64(rest)) / ones
    assert abs(total / 2.0 ** -126 - 1) > 0.1        # far from the limit
    want = scale / k if total >= 2.0 ** -126 else 0.0
    # the scores are equal; the quotient, its product and the scale's round: 2^-22 + 2 * 2^-24.  A score below 2^-126 has
    # fewer bits, the same ones in all eight
    assert np.abs(w[0] - want).max() <= 2.0 ** -21 * scale, (w, want)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [24, 60, 256, 512])
@pytest.mark.parametrize("renormalise", [True, False])
def test_gate_accuracy_of_the_smallest_scores(score, E, renormalise):
    """Experts far below the rest that a bias makes the chosen ones: a score's relative error grows with its logit's distance
    from the largest (a sigmoid's own size), as the argument of its exponential is rounded: 2^-24 of x log2 e, and log2 e
    by 2^-26.2 (7.3e-8 x together); beside it the hardware's exponential and quotient, sums and products: 8 times 2^-23."""
    T, k = 64, 6
    g = torch.Generator().manual_seed(E)
    x = torch.linspace(1.0, 86.0, T)[:, None] + torch.rand(T, k, generator=g) * 0.5     # distances
    logits = torch.zeros(T, E)
    at = torch.randperm(E, generator=g)[:k]
    if score == "softmax":
        logits += 3.0 * torch.rand(T, E, generator=g) - 3.0
        logits[:, (int(at[0]) + 1) % E if (int(at[0]) + 1) % E not in at else next(e for e in range(E) if e not in at)] = 0.0
    logits[:, at] = -x
    bias = torch.zeros(E)
    bias[at] = 4.0 + 2.0 * torch.arange(k, 0, -1).float()
    idx, w = run_gate(logits.cuda(), bias.cuda(), T, E, k, score=score, renormalise=renormalise)
    assert (idx == at.numpy()).all()
    l = logits.double()
    s = (torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1))[:, at]
    normal = (s.amin(1) > 2.0 ** -126).numpy()                # (a score below 2^-126 counts as 0)
    assert normal.mean() > 0.9
    s = (s / s.sum(1, keepdim=True) if renormalise else s).numpy()
    # (renormalised: the sum's error too)
    rel = (7.3e-8 * (x.numpy() + 0.5) + 8 * 2.0 ** -23) * (2 if renormalise else 1)
    assert (np.abs(w - s) <= rel * s)[normal].all(), (np.abs(w - s) / (rel * s))[normal].max()


def test_gate_of_many_tokens():
    """2^20 tokens, and rows whose offsets pass 2^31 elements."""
    T, E, k = 1 << 20, 16, 3
    base = torch.randn(4096, E, generator=torch.Generator().manual_seed(3))
    want = run_gate(base.cuda(), None, 4096, E, k, score="sigmoid")
    for stride in (E, 2304):
        buf = torch.empty(T, stride, dtype=torch.bfloat16 if stride > E else torch.float32, device="cuda")
        buf[:, :E] = base.to(buf.dtype).cuda().repeat(T // 4096, 1)
        if stride > E:
            want = run_gate(base.to(buf.dtype).cuda(), None, 4096, E, k, score="sigmoid")
        idx, w = run_gate(buf, None, T, E, k, stride=stride, score="sigmoid")
        assert (idx.reshape(-1, 4096, k) == want[0]).all() and (w.reshape(-1, 4096, k) == want[1]).all()


@pytest.mark.parametrize("E,k,groups,gk,with_bias,score,dt", [
    (60, 6, 1, 1, False, "softmax", "f16"), (256, 8, 1, 1, False, "sigmoid", "f32"), (256, 8, 8, 4, True, "sigmoid", "f32"),
    (296, 11, 8, 3, False, "sigmoid", "f16"), (512, 32, 1, 1, True, "softmax", "bf16"), (264, 18, 8, 6, False, "softmax", "f32"),
    (1024, 24, 4, 2, True, "sigmoid", "bf16"), (1024, 32, 1, 1, False, "sigmoid", "f32"), (96, 20, 2, 1, False, "softmax", "f32")])
def test_gate_among_many_equals(E, k, groups, gk, with_bias, score, dt):
    """Most logits of a token are one value (or -inf): a few above it, none, more than k, a few below; the choice has to
    be the largest values with the equals in index order."""
    g = torch.Generator().manual_seed(5)
    T = 64
    logits = torch.zeros(T, E)
    logits[1::4] = -torch.inf
    for t in range(T):
        above = [0, 1, k // 2, k - 1, k, k + 3, 40, 2][t % 8]
        at = torch.randperm(E, generator=g)[:min(above + 9, E)]
        logits[t, at[:above]] = (torch.arange(1, E + 1)[:len(at[:above])] % 13 + 1) / 8.0   # ties among them
        logits[t, at[above:]] = -1.0
    logits = logits.to(DT[dt])
    bias = None
    if with_bias:
        bias = (torch.randint(0, 2, (E,), generator=g) * 0.5).float()
    idx, w = run_gate(logits.cuda(), None if bias is None else bias.cuda(), T, E, k, score=score, groups=groups,
                      group_topk=gk, scale=1.0)
    want_idx, want_w, clear = reference(logits.double().numpy(), None if bias is None else bias.numpy(), E, k, score,
                                        groups, gk, "top2", True, 1.0)
    assert clear.all()
    assert np.array_equal(idx, want_idx)
    assert np.abs(w - want_w).max() <= W_RTOL, np.abs(w - want_w).max()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(40, 6), (256, 8), (512, 10)])
def test_gate_of_a_logit_of_minus_infinity_beside_a_bias(E, k, score):
    """Such an expert has a score of 0, so its choice value is its bias: one that is among the k largest takes a slot, with a
    weight of 0; without a bias it comes after every other expert; a bias of -inf keeps it out."""
    T = 20
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(E))
    logits[:, 3] = logits[:, 7] = -np.inf
    bias = torch.zeros(E)
    bias[3], bias[5], bias[7] = 4.0, -np.inf, -np.inf
    idx, w = run_gate(logits.cuda(), bias.cuda(), T, E, k, score=score, renormalise=False)
    assert (idx[:, 0] == 3).all() and (w[:, 0] == 0).all() and (w[:, 1:] > 0).all()
    assert not np.isin(idx, [5, 7]).any()
    idx, w = run_gate(logits.cuda(), None, T, E, k, score=score)
    assert not np.isin(idx, [3, 7]).any()


def test_gate_nan_in_the_bias_switches_the_expert_off():
    l = torch.randn(50, 40, generator=torch.Generator().manual_seed(1))
    b = torch.zeros(40)
    b[7] = float("nan")
    idx, w = run_gate(l.cuda(), b.cuda(), 50, 40, 6, score="sigmoid")
    assert not (idx == 7).any() and np.isfinite(w).all()


@pytest.mark.parametrize("E,k,crowd", [(3, 2, 2), (20, 6, 9), (60, 6, 40), (64, 3, 10), (256, 8, 30), (256, 16, 150),
                                       (1000, 32, 60), (1024, 32, 700)])
@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_compares_the_logits_themselves(E, k, crowd, renormalise, score):
    """Neighbouring fp32 numbers far below a token's largest logit, whose differences from it round to one number, and
    sigmoids that round to 1: the order is that of the logits, to the last bit."""
    T = 16
    g = torch.Generator().manual_seed(E + crowd)
    logits = torch.empty(T, E)
    for t in range(T):
        base, peak = [(1.0, 50.0), (5.0, 20.0), (-0.75, 64.0), (30.0, 30.5)][t % 4]
        near = np.float32(base) + np.arange(crowd, dtype=np.float32) * np.spacing(np.float32(base))
        row = np.full(E, base - 20.0, np.float32)
        at = torch.randperm(E, generator=g).numpy()[:min(E, crowd + 1)]
        row[at[1:]] = near[torch.randperm(crowd, generator=g).numpy()][:len(at) - 1]
        row[at[0]] = peak
        logits[t] = torch.from_numpy(row)
    idx, w = run_gate(logits.cuda(), None, T, E, k, score=score, renormalise=renormalise)
    l = logits.double().numpy()
    want = np.argsort(-l, 1, kind="stable")[:, :k]
    assert np.array_equal(idx, want)
    s = 1.0 / (1.0 + np.exp(-l)) if score == "sigmoid" else np.exp(l - l.max(1, keepdims=True))
    s = np.take_along_axis(s / (s.sum(1, keepdims=True) if score == "softmax" else 1.0), want, 1)
    if renormalise:
        s = s / s.sum(1, keepdims=True)
    # W_RTOL is for |l| + |m| of 32, here up to 65
    assert (np.abs(w - s) <= 2 * W_RTOL * s + 1e-30).all()


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E,k", [(7, 5), (40, 6), (256, 8), (512, 32)])
@pytest.mark.parametrize("renormalise", [True, False])
def test_gate_softmax_of_lowest_and_largest_logits(dt, E, k, renormalise):
    """Masks of the type's lowest value: where they are all a token has they share its weight, before any -inf or NaN;
    beside other logits they count as 0 like these.  Logits of the largest value likewise share."""
    lo, hi = torch.finfo(DT[dt]).min, torch.finfo(DT[dt]).max
    logits = torch.full((6, E), -np.inf)
    logits[0] = lo
    logits[1, E // 2:] = lo
    logits[2, E - 2:] = lo
    logits[2, 0] = float("nan")
    logits[3, ::2] = lo
    logits[3, E - 1] = 1.0
    logits[4] = lo
    logits[4, 1::3] = hi
    logits[5, E - 2] = hi
    idx, w = run_gate(logits.to(DT[dt]).cuda(), None, 6, E, k, renormalise=renormalise)
    for t in range(6):
        l = logits[t].numpy()
        live = np.flatnonzero(l == np.nanmax(l))
        want = (list(live) + [e for e in range(E) if e not in set(live)])[:k]
        assert list(idx[t]) == want, t
        n = min(k, len(live))
        share = 1.0 / (n if renormalise else len(live))
        assert np.abs(w[t][:n] - share).max() <= 2.0 ** -20 * share and (w[t][n:] == 0).all(), t


def by_value(v, count):
    """Order of v, largest first and equals by index, and whether no two different finite values that the first `count`
    places rest on are within what a score's rounding (GAP) could swap."""
    o = sorted(range(len(v)), key=lambda e: (-v[e], e))
    near = any(0 < v[a] - v[b] <= GAP["softmax"] * 2 * abs(v[a]) for a, b in zip(o[:count], o[1:count + 1])
               if np.isfinite(v[a]))
    return o, not near


@pytest.mark.parametrize("E,k,groups,gk", [
    (20, 4, 1, 1), (20, 20, 1, 1), (60, 6, 1, 1), (64, 3, 1, 1), (100, 20, 4, 2), (256, 8, 1, 1), (256, 16, 1, 1),
    (256, 32, 1, 1), (256, 8, 8, 4), (512, 32, 1, 1), (1000, 17, 4, 2), (1020, 32, 17, 9), (1024, 32, 1, 1),
    (1024, 32, 32, 16)])
@pytest.mark.parametrize("score,group_score", [("sigmoid", "top2"), ("softmax", "max")])
def test_gate_infinite_biases(E, k, groups, gk, score, group_score):
    """A bias of +inf forces its expert, however many there are (one, up to all, in more groups than are kept) and
    wherever they lie; of these the lower indices come first.  -inf puts an expert behind the others."""
    T, per = 4, E // groups
    g = torch.Generator().manual_seed(E + k)
    spread = torch.linspace(4.0, -4.0, E)              # distinct scores, thousandths apart
    logits = torch.stack([spread, spread.flip(0), spread[torch.randperm(E, generator=g)],
                          spread[torch.randperm(E, generator=g)]])
    logits[3, ::3] = -np.inf
    s = (torch.sigmoid(logits.double()) if score == "sigmoid" else torch.softmax(logits.double(), 1)).numpy()
    one_per_group = (torch.arange(groups) * per + per // 2).tolist()
    random = torch.randperm(E, generator=g).tolist()
    clear = total = 0
    for forced in ([0], [E - 1], random[:max(1, k - 1)], random[:k], range(E * 2 // 5), range(max(0, E - 16), E),
                   range(E - max(1, k // 2)), range(E), one_per_group, one_per_group[1::2], range(E - per * (groups > 1))):
        for behind in ([], random[E - E // 3:]):
            bias = np.zeros(E)
            bias[list(behind)] = -np.inf
            bias[list(forced)] = np.inf
            idx, w = run_gate(logits.cuda(), torch.tensor(bias, dtype=torch.float32).cuda(), T, E, k, score=score,
                              groups=groups, group_topk=gk, group_score=group_score, renormalise=False)
            for t in range(T):
                v = s[t] + np.maximum(bias, -F32_MAX)  # (-inf counts as the lowest number: its sums stay numbers)
                fine = True
                if groups > 1:
                    top = -np.sort(-v.reshape(groups, per), 1)
                    order, fine = by_value(top[:, 0] if group_score == "max" else np.maximum(top[:, 0] + top[:, 1], -F32_MAX), gk)
                    for dropped in order[gk:]:
                        v[dropped * per:(dropped + 1) * per] = -np.inf
                want, fine2 = by_value(v, k)
                total += 1
                assert len(set(idx[t])) == k and idx[t].min() >= 0 and idx[t].max() < E
                if fine and fine2:
                    clear += 1
                    assert list(idx[t]) == want[:k], (t, list(forced)[:4], len(forced), len(behind))
                    assert (np.abs(w[t] - s[t][want[:k]]) <= W_RTOL * s[t][want[:k]] + 1e-30).all()
    assert clear > 0.9 * total


def test_gate_unaligned_logits_and_zero_tokens():
    l = torch.randn(20, 257, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    view = l[:, 1:]                       # rows at odd elements
    a = run_gate(view, None, 20, 256, 8, stride=257)
    b = run_gate(view.contiguous(), None, 20, 256, 8)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    run_gate(l, None, 0, 256, 8)


def test_gate_on_another_stream():
    s = torch.cuda.Stream()
    l = torch.randn(3000, 256, device="cuda")
    idx = torch.empty(3000, 8, dtype=torch.int32, device="cuda")
    w = torch.empty(3000, 8, device="cuda")
    cfg = moe.gate_config(3000)
    s.wait_stream(torch.cuda.current_stream())
    moe.moe_gate(cfg, l, None, idx, w, stream=s)
    s.synchronize()
    i2, w2 = run_gate(l, None, 3000, 256, 8)
    assert np.array_equal(idx.cpu().numpy(), i2) and np.array_equal(w.cpu().numpy(), w2)


def test_gate_refusal_raises():
    l = torch.zeros(4, 256, device="cuda")
    i = torch.zeros(4, 8, dtype=torch.int32, device="cuda")
    with pytest.raises(moe.MoEError):
        moe.moe_gate(moe.gate_config(4, 256, 8, groups=5, group_topk=2), l, None, i, l)


# ------------------------------------------------------------------------------- moe_dispatch


def layer(T, d=512, I=128):
    wl = configs.custom_workload(f"gate_t{T}", T=T, d=d, I=I)
    shp = moe.shape(T, d, 256, 8, I, I)
    return shp, DeviceLayer(shp, configs.make_layer(wl)), configs.make_x(wl)


@pytest.mark.parametrize("T", [1, 2, 33, 500])
def test_layer_through_the_gate_equals_the_layer_with_its_router(T):
    shp, dl, x = layer(T)
    xd = to_dev(x)
    opts = moe.options(deterministic=1, decode_path=moe.DECODE_GEMV)
    outs, rts = [], []
    for own_router in (True, False):
        rt, ws = moe.Routing(T), moe.workspace(shp, opts)
        y = torch.empty(T, shp.d, dtype=torch.int16, device="cuda")
        for _ in range(2):                 # the second call finds the first one's workspace
            if own_router:
                moe.moe_route(shp, xd, dl.w_router, None, rt, ws, opts)
            else:
                lg = torch.empty(T, 256, device="cuda")
                moe.moe_router_logits(shp, xd, dl.w_router, None, lg)
                moe.moe_gate(moe.gate_config(T), lg, None, rt.topk_idx, rt.topk_w)
                rt.topk_w.copy_(rts[0].topk_w)   # the same weights to the last bit
                moe.moe_dispatch(shp, xd, rt, ws, opts)
            moe.moe_grouped_ffn(shp, xd, rt, dl.packed_routed, dl.packed_shared, ws, opts)
            moe.moe_combine(shp, rt, ws, y, opts)
            rc, bits = moe.moe_read_status(ws)
            assert rc == moe.MOE_OK, bits
        outs.append(y.clone())
        rts.append(rt)
    a, b = rts
    n = int(a.num_tiles.item())
    assert n == int(b.num_tiles.item())
    for f in ("topk_idx", "counts", "offsets", "perm", "pos"):
        assert torch.equal(getattr(a, f), getattr(b, f)), f
    assert torch.equal(a.tiles[:n], b.tiles[:n])
    if T > 1:
        assert torch.equal(outs[0], outs[1])
    else:   # the decode kernels add partial rows with atomics: their order is not fixed
        f = [o.view(torch.bfloat16).float() for o in outs]
        assert (f[0] - f[1]).abs().max() <= 2.0 ** -7 * f[0].abs().max()


def test_dispatch_of_a_skewed_choice():
    """Every token picks expert 255 and seven more; counts, offsets, perm and pos from their definition."""
    T = 333
    shp, dl, x = layer(T)
    rng = np.random.RandomState(0)
    idx = np.stack([np.concatenate([[255], rng.permutation(255)[:7]]) for _ in range(T)]).astype(np.int32)
    rt, ws = moe.Routing(T), moe.workspace(shp)
    rt.topk_idx.copy_(torch.from_numpy(idx))
    rt.topk_w.fill_(0.125)
    moe.moe_dispatch(shp, to_dev(x), rt, ws)
    assert moe.moe_read_status(ws)[0] == moe.MOE_OK
    flat = idx.reshape(-1)
    counts = np.bincount(flat, minlength=256)
    order = np.argsort(flat, kind="stable")
    assert np.array_equal(rt.counts.cpu().numpy(), counts)
    assert np.array_equal(rt.offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(counts)]))
    assert np.array_equal(rt.perm.cpu().numpy(), order)
    pos = np.empty(8 * T, np.int64)
    pos[order] = np.arange(8 * T)
    assert np.array_equal(rt.pos.cpu().numpy().reshape(-1), pos)


def test_dispatch_of_the_largest_chunk():
    T, d = 65536, 256
    shp = moe.shape(T, d, 256, 8, 128, 128)
    x = torch.randint(-100, 100, (T, d), dtype=torch.int16, device="cuda")
    idx = torch.rand(T, 256, device="cuda").argsort(1)[:, :8].int()
    rt, ws = moe.Routing(T), moe.workspace(shp)
    rt.topk_idx.copy_(idx)
    rt.topk_w.fill_(0.125)
    moe.moe_dispatch(shp, x, rt, ws)
    assert moe.moe_read_status(ws)[0] == moe.MOE_OK
    flat = idx.reshape(-1).long()
    counts = torch.bincount(flat, minlength=256)
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(rt.counts.long(), counts) and torch.equal(rt.perm.long(), order)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(8 * T, device="cuda")
    assert torch.equal(rt.pos.reshape(-1).long(), pos)


@pytest.mark.parametrize("T", [1, 40])
def test_dispatch_flags_an_expert_out_of_range(T):
    shp, dl, x = layer(T)
    rt, ws = moe.Routing(T), moe.workspace(shp)
    rt.topk_idx.copy_(torch.arange(8, dtype=torch.int32).repeat(T, 1))
    rt.topk_idx[T - 1, 3] = 256
    rt.topk_idx[0, 5] = -1
    rt.topk_w.fill_(0.125)
    moe.moe_dispatch(shp, to_dev(x), rt, ws)
    rc, bits = moe.moe_read_status(ws)
    assert rc == moe.MOE_ERR_DEVICE_STATUS and bits & moe.MOE_STATUS_BAD_EXPERT
    assert int(rt.counts.sum()) == 8 * T - 2
    pos = rt.pos.cpu().numpy()
    assert pos.min() >= 0 and pos.max() < 8 * T


@pytest.mark.parametrize("deterministic", [0, 1])
@pytest.mark.parametrize("T", [1, 2, 40])
@pytest.mark.parametrize("bad", ["some", "a token", "all"])
def test_an_expert_out_of_range_is_left_out_of_the_sums(T, bad, deterministic):
    """The layer's output is the sum over the valid slots, on a workspace that an earlier call has filled."""
    shp, dl, x = layer(T)
    lay = configs.make_layer(configs.custom_workload(f"gate_t{T}", T=T, d=shp.d, I=shp.I))
    rng = np.random.RandomState(T)
    idx = np.stack([rng.permutation(256)[:8] for _ in range(T)]).astype(np.int32)
    w = rng.uniform(0.05, 0.3, (T, 8)).astype(np.float32)
    off = np.zeros((T, 8), bool)
    off[0, 5] = off[T - 1, 3] = True
    if bad == "a token":
        off[T // 2] = True
    if bad == "all":
        off[:] = True
    opts = moe.options(deterministic=deterministic)
    rt, ws = moe.Routing(T), moe.workspace(shp, opts)
    rt.topk_w.copy_(torch.from_numpy(w))
    xd = to_dev(x)
    for leave_out in (False, True):
        rt.topk_idx.copy_(torch.from_numpy(np.where(off & leave_out, rng.choice([-1, 256, 1 << 30], (T, 8)), idx)))
        y = torch.empty(T, shp.d, dtype=torch.int16, device="cuda")
        moe.moe_dispatch(shp, xd, rt, ws, opts)
        moe.moe_grouped_ffn(shp, xd, rt, dl.packed_routed, dl.packed_shared, ws, opts)
        moe.moe_combine(shp, rt, ws, y, opts)
        rc, bits = moe.moe_read_status(ws)
        assert (rc, bits) == ((moe.MOE_ERR_DEVICE_STATUS, moe.MOE_STATUS_BAD_EXPERT) if leave_out else (moe.MOE_OK, 0))
        ref = oracle.moe_tokens(x, idx, np.where(off & leave_out, 0.0, w.astype(np.float64)), lay.routed, lay.shared)
        assert_output_close(y_to_f64(y), ref, f"left out: {leave_out}")


@pytest.mark.parametrize("T", [1, 100])
def test_the_example_layer(T):
    """examples/gated_layer.py: projections, gate, dispatch and experts of one layer against their formulas."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_layer.py")
    spec = importlib.util.spec_from_file_location("gated_layer", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    layer = ex.GatedLayer(T, d=512, I=128, attention=384, vocab=1000)
    a = torch.randn(T, 384, device="cuda").bfloat16()
    r = torch.randn(T, 512, device="cuda").bfloat16()
    for _ in range(2):
        y, nxt = layer(a, r)
    layer.check_status()
    h = a.double() @ layer.w_out.double().t() + r.double()
    assert ((layer.hidden.double() - h).abs() <= 2.0 ** -8 * h.abs() + 1e-4).all()
    lg = layer.hidden.double() @ layer.w_router.double().t()
    assert ((layer.logits.double() - lg).norm() / lg.norm()).item() <= 1e-6
    ri, rw, clear = reference(layer.logits.cpu().numpy(), layer.balance.cpu().numpy(), 256, 8, "sigmoid", 8, 4, "top2",
                              True, 2.5)
    assert np.array_equal(layer.routing.topk_idx.cpu().numpy()[clear], ri[clear])
    assert ex.compare_with_oracle(layer, list(range(min(T, 8)))) <= 5e-3
    z = layer.y[-nxt.shape[0]:].double() @ layer.w_head.double().t()
    assert ((nxt.double() - z).norm() / z.norm()).item() <= 1e-6
