"""What attention over the paged cache makes of its numbers: how exactly a weight
is kept, scores and values at the ends of their range, infinities.

Tolerances, from the roundings (BF16: half a step, 2^-8 of the value): the
output's, 2^-8 |out|; a weight that the products take as two BF16 values, 2^-8
of what the first leaves, 2^-16 sum w |v|; scores, exponentials and sums in FP32
below 2^-10 sum w |v| (at |score| <= 64: 64 2^-24 from the exponent, head_dim
2^-24 from the sum).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import decode_gemv_byte_amd as nwc  # noqa: E402
from test_gpu_attention import SHAPES, _Batch, _ref_attend, _say  # noqa: E402

pytestmark = pytest.mark.gpu


def _run(b):
    nwc.nwc_attend(b.call())
    torch.cuda.synchronize()


def _reference(b):
    """(out, sum w |v|) in 64 bits of the rows that are no padding."""
    live = torch.from_numpy(b.lengths >= 0).cuda()
    out, size = _ref_attend(b.kp, b.vp, b.table, b.lengths, b.q, b.scale)
    return live, out[live], size[live]


def _check(b, what):
    """Every finite component within the tolerance, every other one the reference's."""
    live, out, size = _reference(b)
    got = b.out[:len(b.lengths)][live].double()
    same = got == out
    assert bool((got.isnan() == out.isnan()).all()), "%s: NaN in other places" % what
    assert bool((same | ~out.isinf()).all()), "%s: other infinities" % what
    err = torch.where(out.isfinite(), (got - out).abs(), 0.0)
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -16 + 2.0 ** -10) * size
    assert bool((err <= tol)[out.isfinite()].all()), "%s: %g over its tolerance" % (what, float((err - tol)[out.isfinite()].max()))


def _slots(b, r):
    """Pages and slots of a row's positions."""
    page = b.kp.shape[2]
    at = np.arange(max(0, int(b.lengths[r])))
    return torch.from_numpy(b.table[r, at // page]).cuda(), torch.from_numpy(at % page).cuda()


@pytest.mark.parametrize("covers", [0, 4000])
@pytest.mark.parametrize("hq,hk,d,page", SHAPES + [(20, 1, 128, 16), (32, 1, 64, 32)])
def test_attend_every_weight_keeps_16_bits(hq, hk, d, page, covers):
    # position p holds 1 in component p alone, so that component is its weight, and no other weight's rounding averages
    # with its own; a weight rounded once would be off by 2^-8 before the output's rounding.  20 rows behind one prefix: blocks
    # of up to 128 columns
    _say("every weight %d %d %d %d %d" % (hq, hk, d, page, covers))
    shared = d // 2 + 3
    lengths = [shared + r % (d - shared) + 1 for r in range(20)] + [d, d - 1, 33, 5, 2, 1]
    b = _Batch(lengths, hq, hk, d, page, [(0, 20, shared)], seed=hq + d, spread=1.5, covers=covers)
    one = torch.eye(d, dtype=torch.bfloat16, device="cuda")
    for r, n in enumerate(lengths):
        pages, slots = _slots(b, r)
        b.vp[pages, :, slots] = one[:n, None].expand(n, hk, d)
    _run(b)
    _check(b, "weights")


@pytest.mark.parametrize("covers", [0, 4000])
@pytest.mark.parametrize("hq,hk,d,page", SHAPES)
def test_attend_scores_of_any_size(hq, hk, d, page, covers):
    # finite scores far from zero: below -1e30 (all equal: the values' mean), above 1e30, and so far apart that the largest
    # takes all, of either sign; keys and queries are powers of two times at most 8 bits, so FP32 holds each score exactly
    _say("scores of any size %d %d %d %d %d" % (hq, hk, d, page, covers))
    b = _Batch([300, 77, 300, 300, 1], hq, hk, d, page, seed=hq * d, covers=covers)
    rnd = np.random.default_rng(d)
    for r, (q, k, steps) in enumerate(((2.0 ** 50, -2.0 ** 50, 0), (2.0 ** 50, 2.0 ** 50, 0), (2.0 ** 18, 2.0 ** 18, 127),
                                       (2.0 ** 18, -2.0 ** 18, 127), (2.0 ** 20, -2.0 ** 20, 0))):
        pages, slots = _slots(b, r)
        b.q[r] = q
        key = k * (1 + rnd.integers(0, steps + 1, int(b.lengths[r])) / 128)
        b.kp[pages, :, slots] = torch.tensor(key, device="cuda").to(torch.bfloat16)[:, None, None].expand(len(key), hk, d)
    _run(b)
    _check(b, "scores")


@pytest.mark.parametrize("covers", [0, 4000])
@pytest.mark.parametrize("hq,hk,d,page", SHAPES + [(20, 1, 128, 16), (32, 1, 64, 32)])
def test_attend_infinite_values(hq, hk, d, page, covers):
    # an infinity among the seen values is its component's result, NaN where two signs meet; the other components keep their
    # exactness, and a padding row inside a group, whose queries may be anything, changes nothing (rows that share a prefix get the
    # same values there, in copied pages too)
    _say("infinite values %d %d %d %d %d" % (hq, hk, d, page, covers))
    lengths = [75, 90, -1, 104, 2, 1, 40, 35, 35, 5, 1] + [640] * 9 + [500, 1300, 64, 333]
    b = _Batch(lengths, hq, hk, d, page, [(0, 7, 70), (7, 11, 17), (11, 20, 600)], seed=hq + d, covers=covers)
    b.q[2] = float("nan")
    b.q[5] = 0
    inf = float("inf")
    for r, n in enumerate(lengths):
        if n > 0:
            pages, slots = _slots(b, r)
            for component, at, value in ((3, 0, inf), (5, n - 1, -inf), (7, 0, -inf), (7, n // 2, inf), (d - 1, n // 3, -inf)):
                b.vp[pages[at], :, slots[at], component] = value
    _run(b)
    live, out, size = _reference(b)
    assert bool(out[:, :, 3].isposinf().all()) and bool(out[:, :, 5].isneginf().all()) and bool(out[:, :, 9].isfinite().all())
    _check(b, "infinite values")
    assert bool((b.out[:len(lengths)][~live] == 7.0).all())


@pytest.mark.parametrize("covers", [0, 4000])
@pytest.mark.parametrize("hq,hk,d,page", SHAPES)
def test_attend_nan_queries_stay_in_their_head(hq, hk, d, page, covers):
    # its output is NaN; the columns beside it, which the same wavefront computes, are as they are without it
    _say("nan queries %d %d %d %d %d" % (hq, hk, d, page, covers))
    b = _Batch([640] * 9 + [75, 33, 1, 1300], hq, hk, d, page, [(0, 9, 600)], seed=hq + d, covers=covers)
    for r, h in ((3, hq // 2), (4, 0), (9, hq - 1), (11, 0), (12, 0)):
        b.q[r, h, d // 3] = float("nan")
    _run(b)
    _check(b, "nan queries")
    assert int(b.out.isnan().sum()) == 5 * d


@pytest.mark.parametrize("covers", [0, 4000])
@pytest.mark.parametrize("hq,hk,d,page", SHAPES + [(20, 1, 128, 16), (32, 1, 64, 32)])
def test_attend_values_at_the_end_of_their_range(hq, hk, d, page, covers):
    # finite values give a finite result: up to the largest, of one sign (whose weighted sum is n times as large) and of both, with
    # flat scores and with scores that grow along the row, so that weights stand above the running maximum; and the smallest
    _say("large values %d %d %d %d %d" % (hq, hk, d, page, covers))
    lengths = [640] * 9 + [75, 1, 33, 1300, 500, 5]
    b = _Batch(lengths, hq, hk, d, page, [(0, 9, 600)], seed=hq + d, covers=covers)
    g = torch.Generator(device="cuda").manual_seed(d)
    most = torch.finfo(torch.bfloat16).max
    v = torch.rand(b.vp.shape, generator=g, device="cuda").mul_(most / 2).add_(most / 2).to(torch.bfloat16)
    v[..., 1::2] *= torch.randint(0, 2, v[..., 1::2].shape, generator=g, device="cuda").mul_(2).sub_(1).to(torch.bfloat16)
    v[..., 4] = most
    v[..., 6] = -most
    v[..., 8:12] *= 2.0 ** -235                                   # 2^-108 and less
    b.vp.copy_(v)
    first = [x[:600] for x in _slots(b, 0)]
    for r in range(1, 9):                                         # the prefix's values, in copied pages too
        pages, slots = (x[:600] for x in _slots(b, r))
        b.vp[pages, :, slots] = b.vp[first[0], :, first[1]]
    for r in (12, 13):                                            # 10 powers of two over the row
        pages, slots = _slots(b, r)
        b.q[r] = 1
        grow = torch.arange(lengths[r], device="cuda") * (10 * 0.6931 / lengths[r] / d / b.scale)
        b.kp[pages, :, slots] = grow.to(torch.bfloat16)[:, None, None].expand(lengths[r], hk, d)
    _run(b)
    assert bool(b.out.isfinite().all())
    _check(b, "large values")


@pytest.mark.parametrize("covers", [0, 4000])
@pytest.mark.parametrize("hq,hk,d,page", SHAPES)
def test_attend_nan_and_infinite_keys(hq, hk, d, page, covers):
    # a NaN key, or an infinite one whose score is +infinity, among a row's own positions or in the prefix: NaN for the heads that
    # see it, whatever else the row holds (an infinite value too), and for no others
    _say("nan keys %d %d %d %d %d" % (hq, hk, d, page, covers))
    b = _Batch([640] * 9 + [75, 33, 1, 1300], hq, hk, d, page, [(0, 9, 600)], seed=hq + d, covers=covers)
    inf = float("inf")
    for r, at, head, value in ((5, 620, 0, float("nan")), (9, 74, hk - 1, float("nan")), (12, 1000, 0, inf), (12, 3, hk - 1, float("nan")),
                               (0, 100, hk // 2, float("nan"))):
        pages, slots = _slots(b, r)
        b.q[r, head * (hq // hk):(head + 1) * (hq // hk), 1] = 1.0
        b.kp[pages[at], head, slots[at], 1] = value
        b.vp[pages[at - 1], head, slots[at - 1], 2] = inf
        if at < 600 and r < 9:                                    # the prefix, in copied pages too
            for x in range(1, 9):
                pages, slots = _slots(b, x)
                b.kp[pages[at], head, slots[at], 1] = value
                b.vp[pages[at - 1], head, slots[at - 1], 2] = inf
    _run(b)
    _check(b, "nan keys")
    assert bool(b.out[0, hk // 2 * (hq // hk)].isnan().all())
