"""Attention of a chunk of new tokens over the paged cache on the GPU, against a
plain 64-bit computation of the same formula.

Tolerance, from the roundings (BF16: half a step, 2^-8 of the value): the output's
own, 2^-8 |out|, and each weight's rounding to BF16, 2^-8 sum w |v|; scores,
exponentials and sums in FP32 stay below a quarter of the latter (at |score| <= 64:
64 2^-24 from the exponent, twice for the rounded product with the maximum,
head_dim 2^-24 from the sum): 2^-10 sum w |v|.
"""
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import decode_gemv_byte_amd as nwc  # noqa: E402

pytestmark = pytest.mark.gpu


def _say(msg):
    print("[gpu-case] " + msg, flush=True)
    sys.stdout.flush()


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Case:
    """A cache, its table and a chunk: new[r] tokens are the last of lengths[r] positions of row r."""

    def __init__(self, new, lengths, hq, hkv, d, page, seed=0, gap=0, interleaved=False, spare=0, front=0):
        g = torch.Generator(device="cuda").manual_seed(seed + d)
        rnd = np.random.default_rng(seed)
        self.new, self.lengths = np.asarray(new), np.asarray(lengths)
        rows = len(new)
        need = np.maximum(1, -(-np.maximum(self.lengths, 1) // page))
        cols = int(need.max()) + spare
        n_pages = int(need.sum()) + 2
        order = rnd.permutation(n_pages)
        self.table = np.full((rows, cols), -1, np.int64)
        at = 0
        for r in range(rows):
            self.table[r, :need[r]] = order[at:at + need[r]]
            at += need[r]
        if interleaved:
            pool = _randn(g, n_pages, 4, hkv, page, d)
            self.k, self.v = pool[:, 1], pool[:, 3]
        else:
            self.k, self.v = _randn(g, n_pages, hkv, page, d), _randn(g, n_pages, hkv, page, d)
        self.page, self.hq, self.hkv, self.d = page, hq, hkv, d
        self.start = front + np.concatenate(([0], np.cumsum(self.new)))
        tokens = int(self.start[-1]) + front
        self.q_all = _randn(g, tokens, hq * d + gap) * 1.5
        self.q = self.q_all[:, :hq * d].view(tokens, hq, d) if not gap else self.q_all.as_strided(
            (tokens, hq, d), (hq * d + gap, d, 1))
        self.out_all = torch.full((tokens, hq * d + gap), 7.0, dtype=torch.bfloat16, device="cuda")
        self.out = self.out_all.as_strided((tokens, hq, d), (hq * d + gap, d, 1))
        self.scale = d ** -0.5

    def call(self, ws=None):
        cache = nwc.PagedCache(self.k, self.v)
        if ws is None:
            ws = torch.full((nwc.nwc_attend_chunk_workspace_size(cache, len(self.new), self.q.shape[0], self.hq),), 255,
                            dtype=torch.uint8, device="cuda")       # NaN, should anything read it unwritten
        self.dev = (_i32(self.table), _i32(self.start), _i32(self.lengths))
        return nwc.AttendChunk(cache, self.dev[0], self.dev[1], self.dev[2], self.q, self.out, ws, scale=self.scale)

    def ref(self, rows=None):
        """(out, sum w |v|) in 64 bits; NaN where nothing is written."""
        tokens, hq, d = self.q.shape
        out = torch.full((tokens, hq, d), float("nan"), dtype=torch.float64, device="cuda")
        size = torch.zeros_like(out)
        s = hq // self.hkv
        for r in range(len(self.new)) if rows is None else rows:
            n, length = int(self.new[r]), int(self.lengths[r])
            if length < 0 or n == 0:
                continue
            length = min(length, self.table.shape[1] * self.page)
            t0 = int(self.start[r])
            at = np.arange(max(length, 1))
            pg = self.table[r, at // self.page]
            ok = torch.from_numpy((pg >= 0) & (pg < self.k.shape[0])).cuda()
            pg = torch.from_numpy(np.clip(pg, 0, self.k.shape[0] - 1)).cuda()
            at = torch.from_numpy(at).cuda()
            pos = length - n + torch.arange(n, device="cuda")
            seen = (at[None] <= pos[:, None]) & ok[None]
            for h in range(self.hkv):
                k, v = (x[pg, h, at % self.page].double() for x in (self.k, self.v))
                for j in range(h * s, (h + 1) * s):
                    score = (self.q[t0:t0 + n, j].double() @ k.T.contiguous()) * self.scale
                    score = torch.where(seen, score, -float("inf"))
                    w = torch.where(seen, torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-1e300)), 0.0)
                    total = w.sum(-1, keepdim=True)
                    w = w / torch.where(total > 0, total, 1.0)
                    used = seen.any(0)                        # slots that nobody sees may hold anything
                    out[t0:t0 + n, j] = w[:, used] @ v[used]
                    size[t0:t0 + n, j] = w[:, used] @ v[used].abs()
        return out, size

    def check(self, what):
        ref, size = self.ref()
        left = ref.isnan()
        got = self.out.double()
        assert bool((got[left] == 7.0).all()), "%s: a row that takes no part was written" % what
        err = torch.where(left, 0.0, (got - ref).abs())
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -10) * size
        bad = ~left & ~(err <= tol)
        assert not bool(bad.any()), "%s: %d of %d outside, worst %g over, first %s" % (
            what, int(bad.sum()), bad.numel(), float((err - tol)[bad].nan_to_num(1e30).max()), bad.nonzero()[0].tolist())
        hidden = self.out_all[:, self.hq * self.d:]
        assert bool((hidden == 7.0).all()), "%s: between the rows" % what


CASES = [  # new tokens, lengths, q heads, kv heads, head_dim, page
    ([1], [1], 1, 1, 64, 16), ([1], [1], 32, 8, 128, 64), ([2], [2], 8, 2, 256, 16), ([1], [700], 10, 5, 192, 32),
    ([5], [512], 32, 8, 128, 64), ([64], [64], 32, 8, 128, 64), ([65], [65], 4, 4, 128, 16), ([33], [40], 28, 4, 128, 16),
    ([130], [1000], 20, 4, 96, 128), ([300], [300], 64, 8, 64, 32), ([257], [1024], 10, 10, 64, 1024),
    ([31, 1, 1, 200, 7], [31, 900, 1, 450, 8], 16, 8, 128, 32), ([1, 0, 3, 0], [77, 5, 3, 0], 16, 1, 128, 16),
    ([100, 17], [100, 2000], 8, 2, 256, 64), ([90, 300], [91, 301], 10, 5, 192, 16), ([3] * 70, list(range(3, 73)), 8, 2, 64, 16),
    ([40], [200], 64, 1, 64, 16), ([19], [119], 35, 1, 96, 64), ([513], [513], 5, 1, 96, 16), ([9], [5000], 40, 1, 128, 64),
    ([1] * 33, [17 * i + 1 for i in range(33)], 32, 8, 128, 16), ([600], [3000], 6, 2, 128, 256)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s-%s-%d-%d-%d-%d" % ((sum(c[0]), max(c[1])) + c[2:]))
@pytest.mark.parametrize("odd", [False, True])
def test_chunk(case, odd):
    _say("chunk %s %s" % (case, odd))
    c = Case(*case, seed=sum(case[0]), gap=8 if odd else 0, interleaved=odd, spare=3 if odd else 0, front=2 if odd else 0)
    call = c.call()
    nwc.nwc_attend_chunk(call)
    torch.cuda.synchronize()
    c.check("first call")
    first = c.out_all.clone()
    nwc.nwc_attend_chunk(call)
    torch.cuda.synchronize()
    assert torch.equal(first, c.out_all)                        # the same bits


@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 8), (96, 12, 4), (128, 32, 8), (192, 4, 2), (256, 6, 1)])
def test_many_items_and_cuts(d, hq, hkv):
    # rows of all lengths around the unit of 64 positions and the items' token counts
    new = [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 5, 1]
    lengths = [64, 65, 31, 32, 64, 128, 127, 65, 1000, 128, 130, 777, 4096, 63]
    _say("many items %s" % ((d, hq, hkv),))
    c = Case(new, lengths, hq, hkv, d, 32, seed=3)
    nwc.nwc_attend_chunk(c.call())
    torch.cuda.synchronize()
    c.check("many")


def test_long_prompt_and_long_context():
    for new, lengths in (([2100], [2100]), ([70], [40000]), ([2, 1500], [20000, 1600])):
        _say("long %s %s" % (new, lengths))
        c = Case(new, lengths, 8, 2, 128, 64, seed=9)
        nwc.nwc_attend_chunk(c.call())
        torch.cuda.synchronize()
        c.check("long")


def test_rows_that_see_nothing_and_padding():
    # row 0: padding; row 1: more tokens than positions; row 2: no positions at all; row 3: ordinary; row 4: past the table
    c = Case([4, 9, 3, 20, 6], [-1, 5, 0, 50, 80], 8, 2, 64, 16, seed=4)
    c.lengths[4] = 10 ** 6                                      # cut to what the table covers
    c.table[4, :] = c.table[4, 0]
    nwc.nwc_attend_chunk(c.call())
    torch.cuda.synchronize()
    got = c.out
    assert bool((got[:4] == 7.0).all())
    assert bool((got[4:8] == 0.0).all()) and bool((got[13:16] == 0.0).all())
    c.lengths[1], c.new[1] = 5, 5
    c.start = c.start.copy()
    ref, size = Case.ref(c, rows=[3, 4])
    for some in (slice(16, 36), slice(36, 42)):
        err = (got[some].double() - ref[some]).abs()
        assert bool((err <= 2.0 ** -8 * ref[some].abs() + (2.0 ** -8 + 2.0 ** -10) * size[some]).all())
    # the tokens of row 1 that see something: positions 0 .. 4
    one = Case([5], [5], 8, 2, 64, 16)
    one.k, one.v, one.table, one.q = c.k, c.v, c.table[1:2], c.q[8:13]
    ref, size = one.ref()
    err = (got[8:13].double() - ref).abs()
    assert bool((err <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -10) * size).all())


def test_starts_that_are_out_of_range_or_descend():
    # device data of any content: nothing outside the tensors is touched, and rows of sound numbers keep their results
    c = Case([6, 5, 7], [20, 30, 40], 4, 2, 64, 16, seed=5)
    ref, size = c.ref()
    # where positions are cut between workgroups follows from all rows, and with it the order of sums: the bits are
    # not those of other starts, but every result is within the tolerance of one
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -10) * size
    for start in ([-5, 6, 11, 18], [0, 6, 11, 10 ** 9], [18, 6, 11, 18]):
        _say("starts %s" % start)
        c.out_all.fill_(7.0)
        c.start = np.asarray(start)
        nwc.nwc_attend_chunk(c.call())
        torch.cuda.synchronize()
        near = ((c.out.double() - ref).abs() <= tol).all(-1).all(-1)
        assert bool(near[6:18].all())
        if start[0] <= 0:
            assert bool(near[:6].all())
        else:
            assert bool((c.out[:6] == 7.0).all())


def test_pages_that_do_not_exist():
    c = Case([40, 70], [200, 300], 8, 2, 128, 16, seed=6)
    c.table[0, 3] = -1
    c.table[0, 12] = 10 ** 8
    c.table[1, 0] = 2 ** 31 - 1
    c.table[1, 18] = -7                                         # the newest tokens' own page
    nwc.nwc_attend_chunk(c.call())
    torch.cuda.synchronize()
    c.check("missing pages")


def test_all_pages_missing_gives_zeros():
    c = Case([3], [50], 4, 4, 64, 16, seed=7)
    c.table[:] = -1
    nwc.nwc_attend_chunk(c.call())
    torch.cuda.synchronize()
    assert bool((c.out == 0).all())


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
def test_slots_behind_the_length_may_hold_anything(d):
    for value in (float("nan"), float("inf"), -float("inf"), 3.3e38):
        c = Case([20, 9], [37, 100], 4, 2, d, 64, seed=8)
        for r in range(2):
            n = int(c.lengths[r])
            pg = int(c.table[r, n // 64])
            c.k[pg, :, n % 64:] = value
            c.v[pg, :, n % 64:] = value
        nwc.nwc_attend_chunk(c.call())
        torch.cuda.synchronize()
        c.check("behind the length %g" % value)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("which", ["k", "v"])
def test_later_tokens_values_do_not_reach_earlier_ones(which, value):
    c = Case([50], [150], 8, 2, 128, 32, seed=10)
    pos = 120                                                   # the 21st new token's
    (c.k if which == "k" else c.v)[int(c.table[0, pos // 32]), 1, pos % 32, 5] = value
    nwc.nwc_attend_chunk(c.call())
    torch.cuda.synchronize()
    got = c.out.clone()
    early = slice(0, 20)
    ref, size = Case([50], [150], 8, 2, 128, 32, seed=10).ref()
    err = (got[early].double() - ref[early]).abs()
    assert bool((err <= 2.0 ** -8 * ref[early].abs() + (2.0 ** -8 + 2.0 ** -10) * size[early]).all())
    # heads of the other key-value head too
    err = (got[:, :4].double() - ref[:, :4]).abs()
    assert bool((err <= 2.0 ** -8 * ref[:, :4].abs() + (2.0 ** -8 + 2.0 ** -10) * size[:, :4]).all())
    late = got[20:, 4:]
    if which == "v":
        want = torch.full_like(late[..., 5], value)
        assert torch.equal(late[..., 5].nan_to_num(1234.0), want.nan_to_num(1234.0))
        others = [i for i in range(128) if i != 5]
        err = (late[..., others].double() - ref[20:, 4:][..., others]).abs()
        tol = 2.0 ** -8 * ref[20:, 4:][..., others].abs() + (2.0 ** -8 + 2.0 ** -10) * size[20:, 4:][..., others]
        assert bool((err <= tol).all())
    elif value != value:
        assert bool(late.isnan().all())
    else:                                                       # scores of +inf (NaN) or -inf (not seen), by the query's sign
        plus = (c.q[20:, 4:, 5] > 0) == (value > 0)
        assert bool(late[plus].isnan().all()) and not bool(late[~plus].isnan().any())


def test_large_scores_and_values():
    # scores far past what a scaled maximum holds exactly, and values whose weighted sums pass FP32's range
    c = Case([40], [300], 4, 2, 64, 32, seed=11)
    c.q *= 2.0 ** 40
    nwc.nwc_attend_chunk(c.call())
    torch.cuda.synchronize()
    # one position wins, or those that tie within FP32's resolution of the scores: outputs are means of values
    assert bool(c.out.isfinite().all()) and float(c.out.abs().max()) <= float(c.v.abs().max())
    k = c.k[torch.from_numpy(c.table[0, :10]).cuda()].transpose(1, 2).reshape(-1, 2, 64)[:300]
    for h in range(4):
        score = c.q[:, h].double() @ k[:, h // 2].double().T
        score[torch.arange(300, device="cuda")[None] > 260 + torch.arange(40, device="cuda")[:, None]] = -float("inf")
        top = score.topk(2, -1)
        clear = top.values[:, 0] - top.values[:, 1] > 64 * 2.0 ** -24 * top.values[:, 0].abs() + 2.0 ** 12
        assert int(clear.sum()) > 30
        v = c.v[torch.from_numpy(c.table[0, :10]).cuda()].transpose(1, 2).reshape(-1, 2, 64)[:300, h // 2]
        assert torch.equal(c.out[clear, h], v[top.indices[clear, 0]])
    c = Case([40], [300], 4, 2, 64, 32, seed=12)
    c.v.fill_(3.0e38)
    nwc.nwc_attend_chunk(c.call())
    torch.cuda.synchronize()
    assert torch.equal(c.out, torch.full_like(c.out, 3.0e38))


def test_captured_call_serves_moving_lengths_and_pages():
    c = Case([1, 40, 3], [10, 60, 200], 8, 2, 128, 16, seed=13, spare=20)
    call = c.call()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    nwc.nwc_attend_chunk(call, stream=stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        nwc.nwc_attend_chunk(call, stream=stream)
    table, start, lengths = c.dev
    rnd = np.random.default_rng(1)
    for new, length in (([1, 40, 3], [10, 60, 200]), ([40, 1, 3], [90, 333, 3]), ([0, 0, 44], [5, 5, 44]), ([14, 15, 15], [14, -1, 100])):
        _say("replay %s %s" % (new, length))
        c.new, c.lengths = np.asarray(new), np.asarray(length)
        c.start = np.concatenate(([0], np.cumsum(c.new)))
        c.table = np.stack([rnd.permutation(c.k.shape[0])[:1].repeat(c.table.shape[1]) for _ in range(3)])
        for r in range(3):
            c.table[r] = rnd.integers(0, c.k.shape[0], c.table.shape[1])
        table.copy_(_i32(c.table))
        start.copy_(_i32(c.start))
        lengths.copy_(_i32(c.lengths))
        c.out_all.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        c.check("replay")
        got = c.out.clone()
        nwc.nwc_attend_chunk(call)
        torch.cuda.synchronize()
        assert torch.equal(got, c.out)


def test_two_calls_on_two_streams():
    a, b = Case([100], [400], 8, 2, 128, 32, seed=14), Case([60, 60], [61, 900], 8, 2, 128, 32, seed=15)
    calls = [x.call() for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(4):
        for call, s in zip(calls, streams):
            nwc.nwc_attend_chunk(call, stream=s)
    torch.cuda.synchronize()
    a.check("first stream")
    b.check("second stream")


def test_a_single_token_agrees_with_nwc_attend():
    lengths = [1, 63, 64, 65, 500]
    c = Case([1] * 5, lengths, 32, 8, 128, 64, seed=16)
    nwc.nwc_attend_chunk(c.call())
    cache = nwc.PagedCache(c.k, c.v)
    out = torch.empty((5, 32, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(nwc.nwc_attend_workspace_size(cache, 5, 32), dtype=torch.uint8, device="cuda")
    nwc.nwc_attend(nwc.Attend(cache, c.dev[0], c.dev[2], c.q, out, ws))
    torch.cuda.synchronize()
    _, size = c.ref()
    # two results, each within its own tolerance
    assert bool(((out.double() - c.out.double()).abs() <= 2.0 ** -7 * out.double().abs() + 2.0 ** -6 * size).all())


def test_more_rows_than_a_workgroup_has_threads():
    rows = 700
    rnd = np.random.default_rng(17)
    new = rnd.integers(0, 4, rows)
    c = Case(new, new + rnd.integers(0, 90, rows), 4, 2, 64, 16, seed=17)
    nwc.nwc_attend_chunk(c.call())
    torch.cuda.synchronize()
    c.check("700 rows")


def test_offsets_past_32_bits():
    # the last page of a cache of more than 2^32 elements a tensor
    n_pages, hkv, page, d = (1 << 32) // (8 * 1024 * 128) + 2, 8, 1024, 128
    _say("cache of %d pages" % n_pages)
    k = torch.zeros((n_pages, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    c = Case([30], [200], 16, 8, 128, 1024, seed=18)
    at = int(c.table[0, 0])
    k[n_pages - 1], v[n_pages - 1] = c.k[at], c.v[at]
    c.k, c.v = k, v
    c.table[0, 0] = n_pages - 1
    nwc.nwc_attend_chunk(c.call())
    torch.cuda.synchronize()
    c.check("far page")


def test_wide_items_and_what_they_do_not_see():
    # rows of more than 192 columns with heads of 128: slots behind the lengths, an inner unit's missing page, tokens that are
    # more than the positions, a padding row, and rows of a token beside them
    for value in (float("nan"), -float("inf"), 3.3e38):
        c = Case([90, 70, 150, 60, 1], [500, 64, 150, 300, 777], 32, 8, 128, 32, seed=21)
        for r in range(5):
            n = int(c.lengths[r])
            if n % 32:
                pg = int(c.table[r, n // 32])
                c.k[pg, :, n % 32:] = value
                c.v[pg, :, n % 32:] = value
        c.table[0, 4] = -1
        c.table[0, 15] = 2 ** 31 - 1
        c.lengths[3] = -1
        call = c.call()
        nwc.nwc_attend_chunk(call)
        torch.cuda.synchronize()
        c.check("wide items, %g behind the lengths" % value)
        first = c.out.clone()
        for _ in range(3):
            nwc.nwc_attend_chunk(call)
            torch.cuda.synchronize()
            assert torch.equal(c.out, first)


def test_wide_items_of_large_values_and_nan_queries():
    c = Case([64, 70], [300, 2000], 32, 8, 128, 64, seed=22)
    c.v.fill_(3.0e38)
    c.q[3, 5, 7] = float("nan")
    c.q[100, 31, 0] = float("inf")
    nwc.nwc_attend_chunk(c.call())
    torch.cuda.synchronize()
    want = torch.full_like(c.out, 3.0e38)
    want[3, 5] = float("nan")
    want[100, 31] = float("nan")
    assert torch.equal(c.out.nan_to_num(1234.0), want.nan_to_num(1234.0))


def test_many_rows_of_some_tokens():
    # heads of 128, more items than are all cut, no long prompt among them
    rnd = np.random.default_rng(23)
    new = rnd.integers(0, 60, 40)
    lengths = new + rnd.integers(1, 300, 40)
    lengths[7] = new[7] // 2                                    # fewer positions than tokens
    c = Case(list(new), list(lengths), 32, 8, 128, 16, seed=24, gap=64)
    for r in range(40):
        n = int(c.lengths[r])
        if n % 16:
            pg = int(c.table[r, n // 16])
            c.k[pg, :, n % 16:] = float("nan")
            c.v[pg, :, n % 16:] = float("inf")
    c.table[3, 0] = -5
    c.lengths[11] = -2
    nwc.nwc_attend_chunk(c.call())
    torch.cuda.synchronize()
    c.check("many rows of some tokens")


def test_refusals_of_device_tensors():
    c = Case([3, 2], [40, 9], 8, 2, 64, 16, seed=25)
    good = c.call()
    cache, (table, start, lengths) = nwc.PagedCache(c.k, c.v), c.dev
    ws = torch.zeros(nwc.nwc_attend_chunk_workspace_size(cache, 2, 5, 8), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c.q)
    for args in ((table, start[:2], lengths, c.q, out, ws), (table, start, lengths[:1], c.q, out, ws), (table, start.long(), lengths, c.q, out, ws),
                 (table, start, lengths, c.q.float(), out, ws), (table, start, lengths, c.q, out[:4], ws), (table, start, lengths, c.q, out, ws.float()),
                 (table, start, lengths, c.q[..., :32], out[..., :32], ws), (table.long(), start, lengths, c.q, out, ws)):
        with pytest.raises(ValueError):
            nwc.AttendChunk(cache, *args)
    odd = torch.zeros((5, 3, 64), dtype=torch.bfloat16, device="cuda")                   # 3 heads for 2 key-value heads
    for bad in (nwc.AttendChunk(cache, table, start, lengths, c.q, c.q, ws), nwc.AttendChunk(cache, table, start, lengths, c.q, out, ws[:256]),
                nwc.AttendChunk(cache, table, start, lengths, odd, odd.clone(), ws),
                nwc.AttendChunk(cache, table, start, lengths, c.q, out, ws, scale=0.0),
                nwc.AttendChunk(cache, table, start, lengths, c.q, out, ws, scale=float("nan")),
                nwc.AttendChunk(cache, table, start, lengths, c.q, out, ws[1:])):
        with pytest.raises(nwc.NwcError):
            nwc.nwc_attend_chunk(bad)
    torch.cuda.synchronize()
    assert bool((c.out == 7.0).all())                           # nothing ran
    nwc.nwc_attend_chunk(good)
    torch.cuda.synchronize()
    c.check("after refusals")
