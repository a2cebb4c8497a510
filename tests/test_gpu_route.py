"""GPU parity of routing, its gradient and the sort of the slots against the oracle.

The choice is compared exactly.  Weights: each is a quotient of float32
exponentials; exp(x - m) carries the rounding of its argument, |x - m| * 2^-24,
and of the function (2 steps), a sum of E such terms (E / 16 + 4) / 2 steps at
most, the quotient and the scale 2 more.  One step is 2^-23, so the relative
error is within (|x - m| / 2 + 8 + E / 32) * 2^-23, with |x - m| up to the row's
spread.  A gradient is a sum of at most top_k + 1 products of such values: the
same relative error, and as many steps, of the sum of their magnitudes, and
half a step of its type where that is bf16.
"""

import math

import numpy as np
import pytest
import torch

from expert_ffn_ragged_amd import rd
from oracle import moe
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(v):
    return torch.tensor([int(v)], dtype=torch.int32, device=DEV)


def logits_of(tokens, experts, dtype, seed, std=1.5):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn((tokens, experts), generator=gen) * std).to(dtype)


def rel_error(x, experts):
    x = x[np.isfinite(x)]
    spread = float(x.max() - min(x.min(), 0.0)) if x.size else 0.0
    return (spread / 2 + 8 + experts / 32) * 2.0 ** -23


CASES = [  # tokens, experts, top_k, groups, top_groups, bias
    (1, 1, 1, 1, 1, False), (1, 2, 2, 1, 1, True), (3, 5, 4, 1, 1, False), (64, 128, 8, 1, 1, False),
    (17, 64, 6, 8, 3, True), (33, 65, 10, 5, 2, True), (40, 256, 8, 8, 4, True), (9, 160, 16, 16, 9, False),
    (21, 257, 3, 1, 1, True), (12, 512, 10, 8, 4, True), (7, 1000, 5, 4, 4, False), (5, 1024, 16, 16, 1, True)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", CASES)
def test_route_and_gradient(case, dtype, score):
    tokens, experts, top_k, groups, top_groups, with_bias = case
    say(f"route {case} {dtype} {score}")
    x = logits_of(tokens, experts, dtype, experts + tokens)
    gen = torch.Generator().manual_seed(7)
    bias = torch.randn((experts,), generator=gen) * 0.1 if with_bias else None
    renorm, scale = tokens % 2 == 1, 2.5 if tokens % 3 == 0 else 1.0
    limit = tokens - tokens // 4
    xd = x.to(DEV)
    w, ids = rd.route(xd, top_k, bias=None if bias is None else bias.to(DEV), score=score, groups=groups,
                      top_groups=top_groups, renormalize=renorm, scale=scale, limit=i32(limit))
    d = torch.randn((tokens, top_k), generator=gen)
    grad = rd.route_bwd(xd, ids, d.to(DEV), score=score, renormalize=renorm, scale=scale)
    torch.cuda.synchronize()
    xv = x.double().numpy()
    want_w, want_ids = moe.route(xv, top_k, None if bias is None else bias.double().numpy(), score, groups, top_groups,
                                 renorm, scale, limit)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    got = w.cpu().double().numpy()
    rel = rel_error(xv, experts)
    assert np.all(np.abs(got - want_w) <= rel * np.abs(want_w)), np.max(np.abs(got - want_w) / np.maximum(want_w, 1e-30))
    want = moe.route_bwd(xv, want_ids, d.double().numpy(), score, renorm, scale)
    assert grad.dtype == dtype
    got = grad.cpu().double().numpy()
    for t in range(tokens):
        p = want_w[t] / scale  # the terms: weight times gradient, and weight times the sum of those
        big = scale * np.abs(d[t].double().numpy())
        mags = np.zeros(experts)
        live = want_ids[t] >= 0
        if score == "softmax" and not renorm:
            s = np.exp(xv[t] - xv[t].max())
            mags += s / s.sum() * (big * p).sum()
        np.add.at(mags, want_ids[t][live], (p * (big + (big * p).sum()))[live])
        tol = (2 * rel + (top_k + 4) * 2.0 ** -23) * mags
        if dtype == torch.bfloat16:
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want[t])
        assert np.all(np.abs(got[t] - want[t]) <= tol), (t, np.max(np.abs(got[t] - want[t]) - tol))
    assert np.all(got[limit:] == 0)


@pytest.mark.parametrize("groups", [1, 4])
def test_ties_go_to_the_lower_expert(groups):
    x = torch.zeros((6, 64))
    x[1, 10:20] = 1.0
    x[2, 63], x[2, 0] = 1.0, 1.0
    x[3] = torch.arange(64) % 3
    x[4, 5], x[4, 6] = -0.0, 0.0
    bias = torch.zeros(64)
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            w, ids = rd.route(x.to(DEV), 8, bias=None if b is None else b.to(DEV), score=score, groups=groups,
                              top_groups=max(1, groups // 2))
            want = moe.route(x.double().numpy(), 8, None if b is None else b.double().numpy(), score, groups,
                             max(1, groups // 2))[1]
            assert np.array_equal(ids.cpu().numpy(), want), (score, b is None)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_close_keys_follow_exact_arithmetic(score):
    """Keys that differ by less than float32 resolves: logits one step apart, biases that nearly cancel."""
    rng = np.random.default_rng(4)
    x = np.float32(rng.normal(size=(200, 64)))
    x[:, 1::2] = np.nextafter(x[:, 0::2], np.float32(9))
    s = 1 / (1 + np.exp(-x[0].astype(np.float64)))
    for bias in (np.zeros(64, np.float32), np.float32(0.5 - s)):
        for groups in (1, 8):
            _, ids = rd.route(torch.from_numpy(x).to(DEV), 6, bias=torch.from_numpy(bias).to(DEV), score=score,
                              groups=groups, top_groups=max(1, groups // 2))
            want = moe.route(x.astype(np.float64), 6, bias.astype(np.float64), score, groups, max(1, groups // 2))[1]
            assert np.array_equal(ids.cpu().numpy(), want), groups


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts", [16, 300])
def test_masked_experts_infinities_and_nan(score, experts):
    inf, nan = math.inf, math.nan
    x = logits_of(8, experts, torch.float32, 3)
    x[0] = -inf
    x[1, 1:] = -inf
    x[2, ::2] = -inf
    x[3] = torch.finfo(torch.float32).min
    x[4, 7] = nan
    x[5, 3] = -300.0
    x[6] = x[6] - 2000.0
    for bias in (None, torch.zeros(experts)):
        for renorm in (False, True):
            for groups in (1, 4):
                kw = dict(score=score, renormalize=renorm, groups=groups, top_groups=max(1, groups // 2))
                w, ids = rd.route(x.to(DEV), 4, bias=None if bias is None else bias.to(DEV), **kw)
                g = rd.route_bwd(x.to(DEV), ids, torch.ones_like(w), score=score, renormalize=renorm)
                want_w, want_ids = moe.route(x.double().numpy(), 4, None if bias is None else bias.numpy(), **kw)
                rows = [0, 1, 2, 3, 5, 6, 7] if score == "softmax" else list(range(8))  # NaN spreads over a softmax
                assert np.array_equal(ids.cpu().numpy()[rows], want_ids[rows]), (renorm, groups)
                got = w.cpu().double().numpy()
                assert np.array_equal(np.isnan(got[rows]), np.isnan(want_w[rows]))
                for t in rows:
                    if not np.isnan(want_w[t]).any():
                        spread = 2000 * 2.0 ** -23 if t == 6 else rel_error(x[t].double().numpy()[:0], experts) * 4
                        np.testing.assert_allclose(got[t], want_w[t], rtol=spread, atol=1e-37)
                assert np.all(got[0] == 0) and np.all(g[0].cpu().numpy() == 0)
                if score == "softmax":
                    assert np.isnan(got[4]).all() and np.all(ids[4].cpu().numpy() >= 0)


def test_gradient_by_differences():
    x = logits_of(5, 40, torch.float32, 8).double()
    d = torch.randn((5, 4), generator=torch.Generator().manual_seed(2))
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            kw = dict(score=score, renormalize=renorm)
            _, ids = rd.route(x.float().to(DEV), 4, **kw)
            g = rd.route_bwd(x.float().to(DEV), ids, d.to(DEV), **kw).cpu().double().numpy()
            xv, h = x.float().double().numpy(), 1e-6
            v = np.random.default_rng(1).normal(size=xv.shape)
            num = ((moe.route(xv + h * v, 4, **kw)[0] - moe.route(xv - h * v, 4, **kw)[0]) * d.numpy()).sum() / (2 * h)
            # the difference quotient: h^2 of the third derivative, 2^-52 / h of the function
            assert abs((g * v).sum() - num) <= 1e-6 * np.abs(g * v).sum() + 1e-8, (score, renorm)


@pytest.mark.parametrize("limit", [-3, 0, 1, 100])
def test_limit_is_clamped_and_outputs_are_whole(limit):
    x = logits_of(20, 30, torch.bfloat16, 1).to(DEV)
    w = torch.full((20, 3), 7.0, device=DEV)
    ids = torch.full((20, 3), 7, dtype=torch.int32, device=DEV)
    x[max(0, limit):] = float("nan")
    rd.route(x, 3, limit=i32(limit), weights=w, ids=ids)
    n = min(max(limit, 0), 20)
    assert torch.all(ids[n:] == -1) and torch.all(w[n:] == 0)
    g = rd.route_bwd(x, ids, torch.ones_like(w))
    assert torch.all(g[n:] == 0)
    want = moe.route(x.cpu().double().numpy(), 3, limit=limit)[1]
    if limit == 1:
        assert np.array_equal(ids.cpu().numpy(), want)


def test_gradient_ignores_ids_outside_the_experts():
    x = logits_of(4, 8, torch.float32, 5).to(DEV)
    ids = torch.tensor([[0, 8], [-1, 3], [2**31 - 1, -2**31], [1, 2]], dtype=torch.int32, device=DEV)
    d = torch.ones((4, 2), device=DEV)
    got = rd.route_bwd(x, ids, d, score="sigmoid").cpu().double().numpy()
    want = moe.route_bwd(x.cpu().double().numpy(), ids.cpu().numpy(), d.cpu().numpy(), "sigmoid")
    np.testing.assert_allclose(got, want, rtol=1e-5, atol=0)
    assert np.all(got[2] == 0)


@pytest.mark.parametrize("n,experts", [(0, 4), (1, 1), (63, 3), (512, 128), (4096, 1024), (4097, 7), (20000, 300),
                                       (131072, 512), (70001, 1024)])
def test_group_rows(n, experts):
    say(f"group_rows {n} {experts}")
    rng = np.random.default_rng(n + experts)
    ids = rng.integers(-1, experts + 1, size=n).astype(np.int32)
    if n > 100:
        ids[:50] = 0
        ids[-30:] = [-2**31, 2**31 - 1] * 15
    sizes, rows, slots, total = rd.group_rows(torch.from_numpy(ids).to(DEV), experts)
    cls = np.where((ids < 0) | (ids >= experts), experts, ids)
    want = np.argsort(cls, kind="stable")
    place = np.empty(n, dtype=np.int64)
    place[want] = np.arange(n)
    assert np.array_equal(rows.cpu().numpy(), want)
    assert np.array_equal(slots.cpu().numpy(), np.where(cls < experts, place, -1))
    assert np.array_equal(sizes.cpu().numpy(), np.bincount(cls, minlength=experts + 1)[:experts])
    assert int(total) == int((cls < experts).sum())


def test_group_rows_matches_the_oracle_and_one_expert_may_take_all():
    rng = np.random.default_rng(0)
    for ids in (rng.integers(-2, 9, size=(37, 4)), np.zeros((60, 8)), np.full((5, 2), -1)):
        ids = ids.astype(np.int32)
        sizes, rows, slots, total = rd.group_rows(torch.from_numpy(ids).to(DEV), 8)
        want = moe.group_rows(ids, 8)
        for got, ref in zip((sizes, rows, slots), want):
            assert np.array_equal(got.cpu().numpy(), ref)
        assert slots.shape == ids.shape and int(total) == want[3]


def test_refusals():
    x = torch.zeros((4, 8), device=DEV)
    with pytest.raises(rd.RDError):
        rd.route(x, 9)
    with pytest.raises(rd.RDError):
        rd.route(x, 2, groups=3)
    with pytest.raises(rd.RDError):
        rd.route(x, 0)
    with pytest.raises(ValueError):
        rd.route(x, 2, score="relu")
    with pytest.raises(ValueError):
        rd.route(x, 2, bias=torch.zeros(7, device=DEV))
    with pytest.raises(TypeError):
        rd.route(x.half(), 2)
    with pytest.raises(ValueError):
        rd.route(x.t(), 2)
    with pytest.raises(ValueError):
        rd.route_bwd(x, torch.zeros((3, 2), dtype=torch.int32, device=DEV), torch.zeros((3, 2), device=DEV))
    with pytest.raises(rd.RDError):
        rd.group_rows(torch.zeros(4, dtype=torch.int32, device=DEV), 0)
    with pytest.raises(rd.RDError):
        rd.group_rows(torch.zeros(100000, dtype=torch.int32, device=DEV), 8,
                      workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("n,experts", [(40 * 4096, 256), (40 * 4096 + 1, 256), (200000, 1024), (3000001, 3)])
def test_group_rows_of_many_workgroups(n, experts):
    """Around the number of workgroups from which their counts are added up beforehand; against torch's stable sort."""
    say(f"group_rows {n} {experts}")
    gen = torch.Generator(device=DEV).manual_seed(n)
    ids = torch.randint(-1, experts + 1, (n,), generator=gen, device=DEV, dtype=torch.int32)
    sizes, rows, slots, total = rd.group_rows(ids, experts)
    inside = (ids >= 0) & (ids < experts)
    key = torch.where(inside, ids, experts).long()
    want = torch.sort(key, stable=True).indices
    assert torch.equal(rows.long(), want)
    assert torch.equal(sizes.long(), torch.bincount(key, minlength=experts + 1)[:experts])
    assert total.item() == int(inside.sum())
    place = torch.empty_like(want)
    place[want] = torch.arange(n, device=DEV)
    assert torch.equal(slots.long(), torch.where(inside, place, -1))



# the float32 bits of four logits near -60, -300 and -650: e^x of the first two add up to less than of the last two,
# by 2^-46.8, 2^-46.2 and 2^-45.4 of the sum (found by a search); the same number of steps added to each keeps that
NEARLY_EQUAL = [(3261884010, 3261746672, 3261898511, 3261738448), (3281412638, 3281401802, 3281441263, 3281390346),
                (3290613656, 3290584961, 3290610543, 3290585567)]


@pytest.mark.parametrize("bits", NEARLY_EQUAL)
def test_nearly_equal_groups_of_small_scores(bits):
    """Two groups of two experts with nearly the same sum of scores, far below a third group's: the choice is that of
    the exact sums.  The interface allows 2^-47 of a score; here sums are off by 2^-50, six roundings of half a step
    each (exponential, reciprocal, sum)."""
    n = 400
    say(f"route nearly equal groups {bits}")
    x = (np.array(bits, np.uint32) + np.arange(n, dtype=np.uint32)[:, None]).view(np.float32)
    e = np.exp(x.astype(np.longdouble))  # sigmoid = e / (1 + e) and softmax = e / sum keep the order of sums of e
    low, high = e[:, 0] + e[:, 1], e[:, 2] + e[:, 3]
    assert np.all(high - low >= 2.0 ** -47 * high) and np.all(high - low <= 2.0 ** -45 * high)
    rows = np.zeros((2 * n, 6), np.float32)
    rows[:n, 2:], rows[n:, 2:] = x, x[:, [2, 3, 0, 1]]
    want = np.repeat([2, 1], n)
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(6, device=DEV)):
            _, ids = rd.route(torch.from_numpy(rows).to(DEV), 4, bias=bias, score=score, groups=3, top_groups=2)
            ids = ids.cpu().numpy()
            assert np.array_equal(ids[:, :2], np.tile([0, 1], (2 * n, 1)))
            assert np.array_equal(ids[:, 2] // 2, want) and np.array_equal(ids[:, 3] // 2, want), (score, bias is None)


@pytest.mark.parametrize("n", [511, 513, 1535, 1536, 1537, 2047, 2048, 2049, 4095])
def test_group_rows_around_the_ids_a_lane_carries(n):
    """One workgroup sorts 512, 1536, 2048 or 4096 ids with 1, 3, 4 or 8 a lane; against a stable sort."""
    for experts in (1, 60, 1024):
        say(f"group_rows {n} {experts}")
        ids = np.random.default_rng(n + experts).integers(-1, experts + 1, size=n).astype(np.int32)
        sizes, rows, slots, total = rd.group_rows(torch.from_numpy(ids).to(DEV), experts)
        cls = np.where((ids < 0) | (ids >= experts), experts, ids)
        want = np.argsort(cls, kind="stable")
        place = np.empty(n, dtype=np.int64)
        place[want] = np.arange(n)
        assert np.array_equal(rows.cpu().numpy(), want)
        assert np.array_equal(slots.cpu().numpy(), np.where(cls < experts, place, -1))
        assert np.array_equal(sizes.cpu().numpy(), np.bincount(cls, minlength=experts + 1)[:experts])
        assert int(total) == int((cls < experts).sum())


def test_counts_are_refused_before_outputs_are_allocated():
    x, ids = torch.zeros((1 << 16, 8), device=DEV), torch.zeros(64, dtype=torch.int32, device=DEV)
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.max_memory_allocated()
    for top_k in (-1, -2**31, 0, 9, 2**31 - 1):
        with pytest.raises(rd.RDError):
            rd.route(x, top_k)
    for experts in (-1, -2**31, 0, 1025, 2**31 - 1):
        with pytest.raises(rd.RDError):
            rd.group_rows(ids, experts)
    with pytest.raises(rd.RDError):
        rd.route(torch.zeros((4, 64), device=DEV), 17)
    assert torch.cuda.max_memory_allocated() < before + (1 << 16)


@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", True)])
@pytest.mark.parametrize("experts,top_k", [(64, 1), (128, 2), (300, 4)])
def test_gradient_of_a_router_that_is_almost_sure(experts, top_k, score, renorm):
    """One expert far above the others: its gradient is the small difference of two nearly equal terms,
    p_i (d_i - sum d p) = p_i (d_i (1 - p_i) - sum of the others' d p), and keeps its relative accuracy.  Each factor
    is a quotient of float32 exponentials, off by rel (see above), three in a product, and a rounding each."""
    say(f"route_bwd almost sure {experts} {top_k} {score} {renorm}")
    tokens = 40
    x = logits_of(tokens, experts, torch.float32, 5 * experts, std=1.0)
    x = x - (14.0 if score == "sigmoid" else 0.0)
    x[torch.arange(tokens), torch.arange(tokens) * 7 % experts] += torch.linspace(4.0, 16.0, tokens)
    d = torch.randn((tokens, top_k), generator=torch.Generator().manual_seed(3))
    xd = x.to(DEV)
    _, ids = rd.route(xd, top_k, score=score, renormalize=renorm)
    got = rd.route_bwd(xd, ids, d.to(DEV), score=score, renormalize=renorm).cpu().double().numpy()
    xv, dv, ids = x.double().numpy(), d.double().numpy(), ids.cpu().numpy()
    want = moe.route_bwd(xv, ids, dv, score, renorm)
    rel = rel_error(xv, experts)
    for t in range(tokens):
        xt, c = xv[t].astype(np.longdouble), ids[t]
        p = np.exp(xt - xt.max()) if score == "softmax" else 1 / (1 + np.exp(-xt))
        p = p / (p[c].sum() if renorm else p.sum())
        mags = np.zeros(experts)
        if not renorm:
            mags += p * (np.abs(dv[t]) * p[c]).sum()
        for i, e in enumerate(c):
            others = sum(abs(dv[t, j]) * p[c[j]] for j in range(top_k) if j != i)
            rest = p[c].sum() - p[e] if renorm else p.sum() - p[e]
            mags[e] = p[e] * (abs(dv[t, i]) * rest + others) * (1 if score == "softmax" else 1 / (1 + np.exp(xt[e])))
        tol = (3 * rel + 4 * 2.0 ** -23) * mags
        assert np.all(np.abs(got[t] - want[t]) <= tol), (t, np.max(np.abs(got[t] - want[t]) - tol))
