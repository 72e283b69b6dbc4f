"""The bins of sample_logits in which a threshold lies: their sums meet every level, whichever threads hold its two sides.

A row's bins are summed by 512 threads, six bins each, in 32 bits, and each thread looks for the level between its own sums.  Sums that a
warp's last thread and the next warp's first form in orders of their own differ in their last bits: a level in between is then found by both,
or by neither.  The sums are restated here as the threads form them."""
import math

import numpy as np
import pytest
import torch

F = np.float32
WARPS, LANES, PER = 16, 32, 6
BINS = WARPS * LANES * PER


def ends(m, handed_on):
    """For bins m [N, BINS]: the sums before and after each bin.  handed_on: a thread begins with the number at which its neighbour ends,
    as the kernel does; otherwise with its own inclusive sum less its own bins."""
    N = m.shape[0]
    m = m.astype(F).reshape(N, WARPS, LANES, PER)
    own = np.zeros((N, WARPS, LANES), F)
    for k in range(0, PER, 2):
        own = own + (m[..., k] + m[..., k + 1])
    upto = own.copy()
    for step in (1, 2, 4, 8, 16):
        other = np.zeros_like(upto)
        other[..., step:] = upto[..., :-step]
        upto = np.where(np.arange(LANES) >= step, upto + other, upto)
    warp = np.zeros((N, WARPS), F)  # the sums of the warps before
    for w in range(1, WARPS):
        for i in range(w):
            warp[:, w] = warp[:, w] + upto[:, i, -1]
    end = warp[:, :, None] + upto
    if handed_on:
        first = np.concatenate([warp[:, :, None], end[..., :-1]], 2)
    else:
        first = upto - own
        for w in range(WARPS):
            for i in range(w):
                first[:, w] = first[:, w] + upto[:, i, -1:]
    before, after = np.empty_like(m), np.empty_like(m)
    at = first
    for k in range(PER):
        before[..., k] = at
        at = end if handed_on and k == PER - 1 else at + m[..., k]
        after[..., k] = at
    return before.reshape(N, BINS), after.reshape(N, BINS)


def rows(kind, N=600):
    rng = np.random.default_rng(7)
    i = np.arange(BINS)
    n = rng.integers(0, 20, (N, BINS)) if kind != "sparse" else (rng.random((N, BINS)) < 0.02) * rng.integers(1, 5, (N, BINS))
    fall = np.exp2(-i / 128) if kind != "flat" else np.exp2(-i / 1e5)
    return (n * fall * rng.uniform(0.7, 1.4, (N, BINS))).astype(F)


@pytest.mark.parametrize("kind", ["dense", "sparse", "flat"])
def test_every_level_is_met(kind):
    m = rows(kind)
    # the restatement sees what it looks for
    before, after = ends(m, False)
    assert (before[:, 1:] < after[:, :-1]).any() and (before[:, 1:] > after[:, :-1]).any()
    # no gap and no overlap
    before, after = ends(m, True)
    assert (before[:, 0] == 0).all() and np.array_equal(before[:, 1:], after[:, :-1])
    # so the first bin up to which there is `lo` and the last one up to which there is `hi` exist, in this order, and the sums lie
    # within 40 roundings of the exact ones: far under the 2^-12 that lies between `lo` and `hi`
    exact = np.cumsum(m.astype(np.float64), 1)
    assert (np.abs(after - exact) <= 40 * 2.0 ** -24 * exact[:, -1:]).all()
    rng = np.random.default_rng(8)
    for r in range(m.shape[0]):
        borders = after[r, PER * LANES - 1::PER * LANES][:-1]
        for level in np.concatenate([rng.uniform(0.01, 0.99, 4) * float(after[r, -1]), borders]).astype(F):
            if level == 0:  # no threshold: something is asked for
                continue
            lo, hi = level * F(1 - 2.0 ** -12), level * F(1 + 2.0 ** -12)
            a = np.flatnonzero((before[r] < lo) & (after[r] >= lo))
            b = np.flatnonzero((before[r] < hi) & (after[r] >= hi))
            assert a.size and (b.size or hi > after[r].max())
            to = b.max() if b.size else BINS - 1
            assert a.min() <= to
            assert (exact[r, a.min() - 1] if a.min() else 0.0) <= level <= exact[r, to] or to == BINS - 1


@pytest.mark.gpu
@pytest.mark.parametrize("N", [2, 30])
@pytest.mark.parametrize("side", [1 - 2.0 ** -12, 1 + 2.0 ** -12])
def test_thresholds_at_the_borders_of_the_warps_bins(side, N):
    """Rows of fp32 in clusters: the level that a threshold's search looks for lies where one warp's bins end."""
    from test_gpu_sample import check, uniforms
    g = torch.Generator().manual_seed(30)
    V = 30011
    x = torch.randn(N, V, generator=g) * 3
    c = math.log2(math.e)
    for w in (1, 2, 3, 5):
        p = []
        for r in range(N):
            y = x[r].double()
            K = round(float(y.max()) * c)
            border = (K + 1 - (w * LANES * PER - 0.5) / 128) / c  # between the last bin of a warp and the next one's first
            mass = torch.exp(y - y.max())
            p.append(float(mass[y >= border].sum() / mass.sum()) / side)
        assert 0.01 < min(p) and max(p) < 1
        outs = [check(x.cuda(), uniforms(torch.Generator().manual_seed(31), N), p=p, exempt=1) for _ in range(3)]
        for o in outs[1:]:
            assert all(torch.equal(o[n], outs[0][n]) for n in o)
