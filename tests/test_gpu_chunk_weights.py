"""How exactly a weight of chunk attention is kept where a token is by itself or a few
are together (at most 32 columns, tokens times query heads of a key-value head).

Position p holds 1 in component p alone, so that component is its weight, and no other
weight's rounding averages with its own.  Tolerance, from the roundings (BF16: half a
step, 2^-8 of the value): the output's, 2^-8 |out|; a weight that the products take as
two BF16 values, 2^-8 of what the first leaves, 2^-16 w; scores, exponentials and sums in
FP32 below 2^-10 w (at |score| <= 64: 64 2^-24 from the exponent, head_dim 2^-24 of sum
|q k| scale from the sum).  A weight rounded once would be off by 2^-8 w before the
output's rounding, and the two together by up to 2^-7 w."""
import numpy as np
import pytest
import torch

from test_gpu_chunk import Case, _say
import decode_gemv_byte_amd as nwc

pytestmark = pytest.mark.gpu


def _weights(c, rows=None):
    """Values of one in each position's own component, for rows of at most head_dim positions."""
    c.v.zero_()
    one = torch.eye(c.d, dtype=torch.bfloat16, device="cuda")
    for r in range(len(c.new)) if rows is None else rows:
        at = np.arange(int(c.lengths[r]))
        pg, slot = torch.from_numpy(c.table[r, at // c.page]).cuda(), torch.from_numpy(at % c.page).cuda()
        c.v[pg, :, slot] = one[:len(at), None].expand(len(at), c.hkv, c.d)


def _check(c, what, rows=None):
    ref, size = c.ref(rows)
    got, own = c.out.double(), ~ref.isnan()
    err, tol = (got - ref).abs(), 2.0 ** -8 * ref.abs() + (2.0 ** -16 + 2.0 ** -10) * size
    bad = own & ~(err <= tol)
    assert not bool(bad.any()), "%s: %d of %d outside, up to %.3g of the weight" % (
        what, int(bad.sum()), int(own.sum()), float((err / size)[bad].max()))


@pytest.mark.parametrize("new", [1, 2, 8])
@pytest.mark.parametrize("hq,hkv,d,page", [(32, 8, 128, 64), (8, 8, 128, 16), (64, 8, 64, 32), (16, 1, 128, 16), (20, 5, 96, 32), (10, 5, 192, 64),
                                           (8, 2, 256, 16), (32, 1, 64, 64)])
def test_every_weight_of_few_columns_keeps_16_bits(hq, hkv, d, page, new):
    new = min(new, 32 * hkv // hq)
    for rows in (1, 13):
        _say("weights of %d rows of %d tokens, %d / %d heads of %d" % (rows, new, hq, hkv, d))
        c = Case([new] * rows, [d - 3 * r for r in range(rows)], hq, hkv, d, page, seed=hq + d + rows)
        _weights(c)
        nwc.nwc_attend_chunk(c.call())
        torch.cuda.synchronize()
        _check(c, "%d rows" % rows)


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (64, 8, 64), (8, 2, 256)])
def test_few_columns_beside_a_prompt(hq, hkv, d):
    # single tokens and three together between parts of prompts: theirs are kept as by themselves
    _say("weights beside prompts, %d / %d heads of %d" % (hq, hkv, d))
    c = Case([1, 300, 3, 1, 40, 1], [d, 700, d - 5, 17, 40, d - 1], hq, hkv, d, 32, seed=d)
    few = [0, 2, 3, 5]
    _weights(c, few)
    nwc.nwc_attend_chunk(c.call())
    torch.cuda.synchronize()
    _check(c, "beside prompts", few)


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (64, 8, 64), (10, 5, 192)])
def test_the_same_token_by_either_attention(hq, hkv, d):
    # a row of one token: nwc_attend_chunk's output is within a rounding of nwc_attend's, at any length
    lengths = [1, 33, 640, 3001, 9000]
    _say("one token by either, %d / %d heads of %d" % (hq, hkv, d))
    c = Case([1] * 5, lengths, hq, hkv, d, 64, seed=2)
    nwc.nwc_attend_chunk(c.call())
    cache = nwc.PagedCache(c.k, c.v)
    ws = torch.empty(nwc.nwc_attend_workspace_size(cache, 5, hq, 0), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c.out)
    nwc.nwc_attend(nwc.Attend(cache, c.dev[0], c.dev[2], c.q, out, ws, scale=c.scale))
    torch.cuda.synchronize()
    _, size = c.ref()
    # each off by its own rounding, half a step of the value, and both by FP32 and the weights' 16 bits
    a, b = c.out.double(), out.double()
    assert bool(((a - b).abs() <= 2.0 ** -8 * (a.abs() + b.abs()) + 2 * (2.0 ** -16 + 2.0 ** -10) * size).all())
    # and hardly ever apart at all.  The weights' 16 bits on both sides, errors of 2^-17 / 3^0.5 each at random, move an output by
    # 2^-17 of what sum w v comes to in the square mean, and a difference crosses a border of rounding as often as it is part of
    # a step, 2^-7.5 of the value between them: 2^-9.5 for values of that size, some times more for smaller ones.  Weights
    # rounded once would move it by 2^-9 of that
    assert float((a != b).double().mean()) < 0.05


def _check_all(c, what):
    """Every finite component within the tolerance, every other one the reference's."""
    ref, size = c.ref()
    got = c.out.double()
    assert bool((got.isnan() == ref.isnan()).all()), "%s: NaN in other places" % what
    assert bool(((got == ref) | ~ref.isinf()).all()), "%s: other infinities" % what
    err, tol = (got - ref).abs(), 2.0 ** -8 * ref.abs() + (2.0 ** -16 + 2.0 ** -10) * size
    bad = ref.isfinite() & ~(err <= tol)
    assert not bool(bad.any()), "%s: %d outside, first %s" % (what, int(bad.sum()), bad.nonzero()[0].tolist())


SOME = [(32, 8, 128), (64, 8, 64), (20, 5, 96), (10, 5, 192), (8, 2, 256)]


@pytest.mark.parametrize("hq,hkv,d", SOME)
def test_infinities_nan_and_large_values_before_few_columns(hq, hkv, d):
    # by one workgroup, and by several whose parts are joined
    new, lengths = [1, 4, 2, 1, 3], [75, 104, 9000, 1, 333]
    most = torch.finfo(torch.bfloat16).max
    for kind in ("infinite", "nan", "largest", "smallest"):
        _say("%s values, %d / %d heads of %d" % (kind, hq, hkv, d))
        c = Case(new, lengths, hq, hkv, d, 32, seed=d)
        if kind in ("largest", "smallest"):
            g = torch.Generator(device="cuda").manual_seed(d)
            c.v.copy_((torch.rand(c.v.shape, generator=g, device="cuda") * 0.5 + 0.5) * (most if kind == "largest" else 2.0 ** -108))
            c.v[..., 1::2] *= torch.randint(0, 2, c.v[..., 1::2].shape, generator=g, device="cuda").mul_(2).sub_(1).to(torch.bfloat16)
        else:
            for r, n in enumerate(lengths):
                at = np.arange(n)
                pg, slot = torch.from_numpy(c.table[r, at // c.page]).cuda(), torch.from_numpy(at % c.page).cuda()
                for e, p, value in ((3, 0, float("inf")), (5, n // 2, -float("inf")), (7, 0, -float("inf")), (7, n // 3, float("inf")),
                                    (d - 1, n - 1, float("inf"))) if kind == "infinite" else ((3, 0, float("nan")), (9, n - 1, float("nan"))):
                    c.v[pg[p], :, slot[p], e] = value
        nwc.nwc_attend_chunk(c.call())
        torch.cuda.synchronize()
        if kind in ("infinite", "nan"):
            # what a token does not see may be infinite or NaN too; the reference multiplies it by zero: component by component
            ref, size = c.ref()
            for r, n in enumerate(lengths):
                t0, own = int(c.start[r]), n - int(c.new[r])
                for i in range(int(c.new[r])):
                    seen = own + i + 1
                    one = Case([1], [seen], hq, hkv, d, c.page)
                    one.k, one.v, one.table, one.q = c.k, c.v, c.table[r:r + 1], c.q[t0 + i:t0 + i + 1]
                    ref[t0 + i:t0 + i + 1], size[t0 + i:t0 + i + 1] = one.ref()
            c.ref = lambda: (ref, size)
        _check_all(c, kind)


@pytest.mark.parametrize("hq,hkv,d", SOME)
def test_scores_of_any_size_before_few_columns(hq, hkv, d):
    # finite scores far from zero, all equal or so far apart that the largest takes all; keys and queries are powers of two times
    # at most 8 bits, so that FP32 holds each score exactly
    _say("scores of any size, %d / %d heads of %d" % (hq, hkv, d))
    lengths = [300, 77, 300, 3000, 1]
    c = Case([1, 2, 3, 1, 1], lengths, hq, hkv, d, 32, seed=d + 1)
    rnd = np.random.default_rng(d)
    for r, (q, k, steps) in enumerate(((2.0 ** 50, -2.0 ** 50, 0), (2.0 ** 50, 2.0 ** 50, 0), (2.0 ** 18, 2.0 ** 18, 127),
                                       (2.0 ** 18, -2.0 ** 18, 127), (2.0 ** 20, -2.0 ** 20, 0))):
        at = np.arange(lengths[r])
        pg, slot = torch.from_numpy(c.table[r, at // c.page]).cuda(), torch.from_numpy(at % c.page).cuda()
        c.q[int(c.start[r]):int(c.start[r + 1])] = q
        key = torch.tensor(k * (1 + rnd.integers(0, steps + 1, lengths[r]) / 128), device="cuda").to(torch.bfloat16)
        c.k[pg, :, slot] = key[:, None, None].expand(lengths[r], hkv, d)
    nwc.nwc_attend_chunk(c.call())
    torch.cuda.synchronize()
    _check_all(c, "scores")
