"""Norm and rotation of heads, the append to a paged cache and attention over it
on the GPU, against plain 64-bit computations of the same formulas.

Tolerances, from the roundings (BF16: half a step, 2^-8 of the value):
 * heads: the result is rounded once, 2^-8 |out|; before it, FP32 arithmetic
   (about ten roundings of 2^-24) and the hardware's sine and cosine, allowed
   2^-17 each, on the pair's two components: 2^-16 (|a| + |b|).
 * attention: the output's rounding, 2^-8 |out|, and each weight's rounding to
   BF16, 2^-8 sum w |v|; scores, exponentials and sums in FP32 stay below a
   quarter of that together (at |score| <= 64: 64 2^-24 from the exponent,
   head_dim 2^-24 from the sum): 2^-10 sum w |v|.
"""
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import decode_gemv_byte_amd as nwc  # noqa: E402

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _say(msg):
    print("[gpu-case] " + msg, flush=True)
    sys.stdout.flush()


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _freqs(dims, base=10000.0):
    return (base ** (-torch.arange(0, dims, 2, dtype=torch.float64) / dims)).float().cuda() if dims else None


def _ref_heads(x, weight, positions, freqs, style, eps=EPS):
    """(result, |a| + |b| of each component's pair) in 64 bits."""
    x = x.double()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    out, size = x.clone(), x.abs()
    if freqs is not None:
        n = freqs.numel()
        i, j = (slice(0, n), slice(n, 2 * n)) if style == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
        phi = positions.double()[:, None, None] * freqs.double()
        a, b = x[..., i], x[..., j]
        out[..., i], out[..., j] = a * phi.cos() - b * phi.sin(), b * phi.cos() + a * phi.sin()
        size[..., i] = size[..., j] = a.abs() + b.abs()
    return out, size


def _check_heads(got, ref, size, what):
    err = (got.double() - ref).abs()
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -16 * size
    assert bool((err <= tol).all()), "%s: %g over its tolerance" % (what, float((err - tol).max()))


HEAD_CASES = [  # tokens, q heads, k heads, head_dim, dims, style, norm
    (1, 32, 8, 128, 128, "half", True), (1, 1, 1, 8, 0, "half", True), (5, 3, 0, 16, 16, "pairs", False),
    (7, 5, 2, 64, 32, "half", True), (33, 28, 4, 128, 64, "pairs", True), (3, 20, 4, 96, 96, "half", False),
    (130, 2, 1, 40, 32, "half", True), (11, 10, 5, 192, 96, "pairs", True), (2, 8, 2, 256, 256, "half", True),
    (9, 0, 7, 80, 80, "half", True), (1000, 32, 8, 128, 128, "half", True), (601, 16, 1, 112, 48, "half", True),
    (1024, 7, 3, 248, 16, "pairs", False), (4, 3, 3, 72, 0, "pairs", False), (6, 4, 2, 128, 24, "half", True),
    (300, 5, 5, 64, 8, "half", False), (70, 9, 1, 200, 200, "half", True), (5000, 9, 3, 64, 40, "pairs", True)]


@pytest.mark.parametrize("case", HEAD_CASES, ids=lambda c: "-".join(map(str, c)))
def test_norm_rope(case):
    t, hq, hk, d, dims, style, norm = case
    _say("norm_rope %s" % (case,))
    g = torch.Generator(device="cuda").manual_seed(t * 1000 + d)
    ld = (hq + hk) * d + 8                                     # a joint projection's rows, with a gap
    x = _randn(g, t, ld) * 3
    q = x[:, :hq * d].view(t, hq, d) if hq else None
    k = x[:, hq * d:(hq + hk) * d].view(t, hk, d) if hk else None
    w = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) if norm else None for _ in range(2)]
    pos = _i32(np.random.default_rng(t).integers(0, 5000, t))
    pos[t // 2] = 2 ** 31 - 1                                  # the farthest position
    if t > 2:
        pos[t - 1] = -1                                        # padding
    freqs = _freqs(dims)
    outs = [None if s is None else torch.full_like(s, 7.0).contiguous() for s in (q, k)]
    before = x.clone()
    nwc.nwc_qk_norm_rope(nwc.QkNormRope(q, k, pos, q_out=outs[0], k_out=outs[1], q_weight=w[0], k_weight=w[1], eps=EPS,
                                        freqs=freqs, style=style))
    torch.cuda.synchronize()
    assert torch.equal(x, before)
    live = (pos >= 0).nonzero()[:, 0]
    for name, src, out, wt in (("q", q, outs[0], w[0]), ("k", k, outs[1], w[1])):
        if src is not None:
            ref, size = _ref_heads(src[live], wt, pos[live], freqs, style)
            _check_heads(out[live], ref, size, name)
            assert bool((out[pos < 0] == 7.0).all()), "padding was written"
    # in place, the gap between the rows untouched
    nwc.nwc_qk_norm_rope(nwc.QkNormRope(q, k, pos, q_weight=w[0], k_weight=w[1], eps=EPS, freqs=freqs, style=style))
    torch.cuda.synchronize()
    for src, out in ((q, outs[0]), (k, outs[1])):
        if src is not None:
            assert torch.equal(src[live], out[live])
    assert torch.equal(x[:, (hq + hk) * d:], before[:, (hq + hk) * d:])
    if t > 2:
        assert torch.equal(x[-1], before[-1])


def test_norm_rope_more_tokens_than_a_launch_has_wavefronts():
    t, d = (1 << 26) + 5, 8
    _say("norm_rope %d tokens of one head of %d" % (t, d))
    g = torch.Generator(device="cuda").manual_seed(26)
    x = torch.empty((t, 1, d), dtype=torch.bfloat16, device="cuda").uniform_(-2, 2, generator=g)
    w = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).clamp(0, 2).to(torch.bfloat16)
    pos = torch.arange(t, dtype=torch.int32, device="cuda") % 4096
    freqs = _freqs(d)
    out = torch.full_like(x, 7.0)
    nwc.nwc_qk_norm_rope(nwc.QkNormRope(x, None, pos, q_out=out, q_weight=w, eps=EPS, freqs=freqs))
    torch.cuda.synchronize()
    for first in (0, 1 << 22, 1 << 24, (1 << 26) - 1000, t - 4096):
        some = slice(first, min(first + 4096, t))
        ref, size = _ref_heads(x[some], w, pos[some], freqs, "half")
        _check_heads(out[some], ref, size, "tokens from %d" % first)
    # a normed head of 8 has length sqrt 8, so a turned pair of it, weighted by at most 2, stays below 6
    assert not bool((out == 7.0).any()), "a token was left out"


def test_norm_rope_special_values():
    # a head of zeros stays zero; infinities and NaN stay in their head; large and tiny values keep the norm's range
    x = torch.ones((6, 1, 64), dtype=torch.bfloat16, device="cuda")
    x[0] = 0
    x[1, 0, 3] = float("nan")
    x[2, 0, 5] = float("inf")
    x[3] *= 2.0 ** 60
    x[4] *= 2.0 ** -60
    pos = _i32([0, 1, 2, 0, 0, 9])
    out = torch.empty_like(x)
    one = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    nwc.nwc_qk_norm_rope(nwc.QkNormRope(x, None, pos, q_out=out, q_weight=one, eps=EPS, freqs=_freqs(32)))
    torch.cuda.synchronize()
    assert bool((out[0] == 0).all())
    assert bool(out[1].isnan().all())                          # the norm is NaN
    assert bool(out[2].isnan().any())                          # inf / inf
    # 2^60: the mean of squares is 2^120, in range: ones; 2^-60: eps rules, 2^-60 / 1e-3
    assert torch.equal(out[3], torch.ones_like(out[3]))
    ref, size = _ref_heads(x[4:], one, pos[4:], _freqs(32), "half")
    _check_heads(out[4:], ref, size, "tiny and ordinary")


def _pages(g, n, h, page, d, interleaved=False):
    if interleaved:                                            # keys and values of two layers in one allocation
        both = _randn(g, n, 4, h, page, d)
        return both[:, 2], both[:, 3]
    return _randn(g, n, h, page, d), _randn(g, n, h, page, d)


APPEND_CASES = [  # sequences, most new tokens, context, q heads, kv heads, head_dim, page, dims, style, norm
    (1, 1, 0, 32, 8, 128, 64, 128, "half", True), (1, 1, 15, 0, 1, 64, 16, 64, "pairs", False),
    (5, 1, 100, 28, 4, 128, 32, 64, "half", True), (3, 40, 9, 8, 2, 256, 16, 256, "half", True),
    (4, 70, 63, 20, 4, 96, 128, 48, "pairs", True), (2, 600, 5, 0, 5, 192, 64, 0, "half", False),
    (2, 33, 31, 3, 3, 40, 1024, 32, "half", True)]


@pytest.mark.parametrize("case", APPEND_CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(case, interleaved):
    n, new, context, hq, hk, d, page, dims, style, norm = case
    _say("append %s %s" % (case, interleaved))
    g = torch.Generator(device="cuda").manual_seed(d + new)
    rnd = np.random.default_rng(new)
    counts = rnd.integers(1, new + 1, n)
    rows = np.repeat(np.arange(n), counts)
    positions = np.concatenate([context + np.arange(c) for c in counts])
    order = rnd.permutation(len(rows))                         # tokens in any order
    rows, positions = rows[order], positions[order]
    cols = -(-(context + new) // page)
    n_pages = n * cols + 3
    table = rnd.permutation(n_pages)[:n * cols].reshape(n, cols)
    kp, vp = _pages(g, n_pages, hk, page, d, interleaved)
    t = len(rows)
    x = _randn(g, t, (hq + 2 * hk) * d) * 2
    q = x[:, :hq * d].view(t, hq, d) if hq else None
    k, v = x[:, hq * d:(hq + hk) * d].view(t, hk, d), x[:, (hq + hk) * d:].view(t, hk, d)
    w = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) if norm else None for _ in range(2)]
    q_out = torch.full_like(q, 7.0).contiguous() if hq else None
    freqs = _freqs(dims)
    positions = positions.copy()
    drop = []
    if t > 3:
        positions[1] = -5                                      # padding
        rows = rows.copy()
        rows[2] = n                                            # no such row
        positions[3] = cols * page                             # past the table
        drop = [1, 2, 3]
        if cols > 1 and t > 6:                                 # pages that do not exist
            table = table.copy()
            drop += [i for i in range(t) if i not in drop and rows[i] == 0 and positions[i] // page == cols - 1]
            table[0, cols - 1] = n_pages
    k0, v0 = kp.clone(), vp.clone()
    if n == 1 and new == 1:
        call_rows = None
    else:
        call_rows = _i32(rows)
    nwc.nwc_kv_append(nwc.KvAppend(nwc.PagedCache(kp, vp), _i32(table), k, v, _i32(positions), rows=call_rows,
                                   k_weight=w[1], q=q, q_out=q_out, q_weight=w[0] if hq else None, eps=EPS, freqs=freqs,
                                   style=style))
    torch.cuda.synchronize()
    keep = np.array([i for i in range(t) if i not in drop])
    pos_all = _i32(np.maximum(positions, 0))
    kr, ks = _ref_heads(k, w[1], pos_all, freqs, style)
    touched = torch.zeros(kp.shape[:3], dtype=torch.bool, device="cuda")
    if len(keep):
        pg, sl = torch.from_numpy(table[rows[keep], positions[keep] // page]).cuda(), torch.from_numpy(positions[keep] % page).cuda()
        idx = torch.from_numpy(keep).cuda()
        _check_heads(kp[pg, :, sl], kr[idx], ks[idx], "keys")
        assert torch.equal(vp[pg, :, sl], v[idx])
        touched[pg, :, sl] = True
    assert torch.equal(kp[~touched], k0[~touched]) and torch.equal(vp[~touched], v0[~touched])
    if hq:
        live = _i32(positions) >= 0
        qr, qs = _ref_heads(q, w[0], pos_all, freqs, style)
        _check_heads(q_out[live], qr[live], qs[live], "queries")
        assert bool((q_out[~live] == 7.0).all())


def _ref_attend(kp, vp, table, lengths, q, scale):
    """(out, sum w |v|) in 64 bits; positions on pages that do not exist are not seen."""
    B, hq, d = q.shape
    n_pages, hk, page, _ = kp.shape
    out = torch.zeros((B, hq, d), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(out)
    for r in range(B):
        n = min(int(lengths[r]), table.shape[1] * page)
        if n <= 0:
            continue
        at = np.arange(n)
        pg = table[r, at // page]
        ok = (pg >= 0) & (pg < n_pages)
        pg, sl = torch.from_numpy(pg[ok].astype(np.int64)).cuda(), torch.from_numpy(at[ok] % page).cuda()
        if not len(pg):
            continue
        k, v = (x[pg, :, sl].double() for x in (kp, vp))        # [n, hk, d]
        for h in range(hk):
            s = hq // hk
            w = torch.softmax(q[r, h * s:(h + 1) * s].double() @ k[:, h].T.contiguous() * scale, -1)
            out[r, h * s:(h + 1) * s] = w @ v[:, h].contiguous()
            size[r, h * s:(h + 1) * s] = w @ v[:, h].abs().contiguous()
    return out, size


def _check_attend(got, ref, what):
    out, size = ref
    err = (got.double() - out).abs()
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2.0 ** -10) * size
    assert bool((err <= tol).all()), "%s: %g over its tolerance" % (what, float((err - tol).max()))


class _Batch:
    """Rows of `lengths` tokens over a fresh cache; groups: (first row, end, shared length)."""

    def __init__(self, lengths, hq, hk, d, page, groups=(), seed=0, interleaved=False, spread=1.0, extra=2, covers=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = np.random.default_rng(seed)
        self.lengths = np.asarray(lengths)
        B = len(lengths)
        cols = -(-max(int(self.lengths.max()), 1, covers) // page)
        need = np.maximum(0, -(-self.lengths // page))
        n_pages = int(need.sum()) + 5 + sum(-(-s // page) for _, _, s in groups)
        free = list(rnd.permutation(n_pages))
        self.kp, self.vp = _pages(g, n_pages, hk, page, d, interleaved)
        table = np.full((B, cols), -1, np.int64)
        for r in range(B):
            for j in range(need[r]):
                table[r, j] = free.pop()
        for first, end, s in groups:
            rows = [r for r in range(first, end) if self.lengths[r] >= s]
            for r in rows[1:]:                                  # whole pages shared, the page that s ends in copied
                table[r, :s // page] = table[rows[0], :s // page]
                if s % page:
                    a, b = table[r, s // page], table[rows[0], s // page]
                    self.kp[a, :, :s % page], self.vp[a, :, :s % page] = self.kp[b, :, :s % page], self.vp[b, :, :s % page]
        # what no row sees may be anything
        seen = torch.zeros((n_pages, page), dtype=torch.bool)
        for r in range(B):
            at = np.arange(max(0, self.lengths[r]))
            seen[table[r, at // page], at % page] = True
        seen = seen.cuda()[:, None, :, None]
        self.kp.masked_fill_(~seen, float("nan"))
        self.vp.masked_fill_(~seen, float("inf"))
        self.q = _randn(g, B, hq, d) * spread
        self.table, self.scale = table, d ** -0.5
        self.groups = (_i32([f for f, _, _ in groups] + [groups[-1][1]]), _i32([s for _, _, s in groups])) if groups else (None, None)
        self.out = torch.full((B + extra, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
        self.cache = nwc.PagedCache(self.kp, self.vp)
        self.ws = torch.full((nwc.nwc_attend_workspace_size(self.cache, B, hq, len(groups)),), 255, dtype=torch.uint8, device="cuda")

    def call(self, groups=True, out=None):
        gs, sl = self.groups if groups else (None, None)
        return nwc.Attend(self.cache, _i32(self.table), _i32(self.lengths), self.q,
                          self.out[:len(self.lengths)] if out is None else out, self.ws, self.scale, gs, sl)

    def check(self, what):
        B = len(self.lengths)
        live = torch.from_numpy(self.lengths >= 0).cuda()
        out, size = _ref_attend(self.kp, self.vp, self.table, self.lengths, self.q, self.scale)
        _check_attend(self.out[:B][live], (out[live], size[live]), what)
        assert bool((self.out[:B][~live] == 7.0).all()) and bool((self.out[B:] == 7.0).all()), "rows that are none were written"


SHAPES = [(32, 8, 128, 64), (28, 4, 128, 16), (64, 8, 64, 32), (8, 1, 256, 16), (20, 4, 96, 128), (10, 5, 192, 32),
          (40, 1, 128, 16), (64, 1, 64, 64), (3, 3, 64, 1024), (33, 1, 256, 32)]


@pytest.mark.parametrize("covers", [0, 2049, 20000])            # tables as long as the rows, and longer ones
@pytest.mark.parametrize("hq,hk,d,page", SHAPES)
def test_attend_ragged(hq, hk, d, page, covers):
    _say("attend ragged %d %d %d %d %d" % (hq, hk, d, page, covers))
    b = _Batch([1, 0, 31, 32, 33, -1, 64, 65, 127, 129, 300, 1000, 16, 17, 2, -7], hq, hk, d, page, seed=d + hq, covers=covers)
    nwc.nwc_attend(b.call())
    torch.cuda.synchronize()
    b.check("ragged")
    assert bool((b.out[1] == 0).all())                         # nothing to see: zeros


@pytest.mark.parametrize("covers", [0, 4096])
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 511, 512, 513, 5000, 40001])
def test_attend_single(length, covers):
    _say("attend single %d %d" % (length, covers))
    b = _Batch([length], 32, 8, 128, 64, seed=length, interleaved=length % 2 == 1, covers=covers)
    nwc.nwc_attend(b.call())
    torch.cuda.synchronize()
    b.check("single")


GROUPS = {
    "one": ([130, 100, 97, 96, 2000], [(0, 5, 96)]),
    "unaligned": ([130, 100, 97, 2000, 91, 90], [(0, 6, 90)]),              # the last row ends with the prefix
    "short rows": ([50, 0, -1, 700, 640, 33, 639, 900], [(0, 8, 640)]),       # rows shorter than the prefix
    "several": ([100] * 3 + [300] * 9 + [41] + [500] * 20, [(0, 3, 77), (3, 12, 256), (12, 13, 40), (13, 33, 450)]),
    "large": (list(range(1200, 1290)), [(0, 90, 1100)]),
    "nothing shared": ([10, 20], [(0, 2, 0)]),
    "shared is all": ([64, 64, 64], [(0, 3, 64)]),
}


@pytest.mark.parametrize("covers", [0, 5000])                     # short tables take a launch of their own
@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("hq,hk,d,page", [SHAPES[0], SHAPES[1], SHAPES[3], SHAPES[4], SHAPES[5], SHAPES[7]])
def test_attend_groups(name, hq, hk, d, page, covers):
    _say("attend groups %s %d %d %d %d %d" % (name, hq, hk, d, page, covers))
    lengths, groups = GROUPS[name]
    b = _Batch(lengths, hq, hk, d, page, groups, seed=len(lengths) + d, covers=covers)
    nwc.nwc_attend(b.call())
    torch.cuda.synchronize()
    b.check(name)
    first = b.out.clone()
    nwc.nwc_attend(b.call(groups=False))                        # each row by itself: the same but for rounding
    torch.cuda.synchronize()
    b.check(name + ", no groups")
    b.out.fill_(7.0)
    b.ws.fill_(0)
    nwc.nwc_attend(b.call())
    torch.cuda.synchronize()
    assert torch.equal(b.out, first), "not the same bits"


@pytest.mark.parametrize("covers", [0, 4000])
def test_attend_any_group_numbers(covers):
    # starts out of order or range, lengths negative or too long: never out of bounds; since all rows have the same pages,
    # whatever is read once is right for every row
    lengths = [200] * 12
    b = _Batch(lengths, 8, 2, 64, 16, [(0, 12, 192)], seed=3, covers=covers)
    for start, shared in (([-5, 4, 100], [192, 64]), ([8, 2, 12], [192, 100]), ([0, 20, 3], [10 ** 9, -4]),
                          ([12, 12, 12], [5, 5]), ([-2 ** 31, 2 ** 31 - 1, 0], [128, 128])):
        _say("any group numbers %s %s" % (start, shared))
        b.groups = (_i32(start), _i32(shared))
        b.ws = torch.empty(nwc.nwc_attend_workspace_size(b.cache, 12, 8, 2), dtype=torch.uint8, device="cuda")
        b.out.fill_(7.0)
        nwc.nwc_attend(b.call())
        torch.cuda.synchronize()
        b.check(str(start))


@pytest.mark.parametrize("covers", [0, 4000])
def test_attend_pages_that_do_not_exist(covers):
    b = _Batch([300, 64, 500], 8, 2, 128, 16, seed=5, covers=covers)
    n = b.kp.shape[0]
    b.table[0, 2], b.table[0, 18], b.table[2, 0], b.table[2, 7] = -1, n, 2 ** 31 - 1, -2 ** 31
    b.table[1, :4] = -1                                         # the whole row
    nwc.nwc_attend(b.call())
    torch.cuda.synchronize()
    b.check("missing pages")
    assert bool((b.out[1] == 0).all())
    b.lengths = np.array([2 ** 31 - 1, 64, 500])                # longer than the table: cut to it
    b.table[0] = np.where(b.table[0] < 0, 0, b.table[0]) % n
    b.kp.copy_(torch.nan_to_num(b.kp, nan=0.5))
    b.vp.copy_(torch.nan_to_num(b.vp, posinf=0.5))
    nwc.nwc_attend(b.call())
    torch.cuda.synchronize()
    b.check("cut")


@pytest.mark.parametrize("covers", [0, 4000])
def test_attend_sharp_and_flat_softmax(covers):
    # scores far apart (one position takes all), all equal, growing along the row (the running maximum moves in every
    # unit), and an infinite one
    b = _Batch([700, 700, 700], 4, 1, 64, 32, seed=8, spread=30.0, covers=covers)
    b.q[1] = 0
    t = torch.from_numpy(b.table).cuda()
    at = torch.arange(700, device="cuda")
    b.q[2] = 1
    b.kp[t[2, at // 32], :, at % 32] = (at / 100).to(torch.bfloat16)[:, None, None].expand(700, 1, 64)
    nwc.nwc_attend(b.call())
    torch.cuda.synchronize()
    out, size = _ref_attend(b.kp, b.vp, b.table, b.lengths, b.q, b.scale)
    err = (b.out[:3].double() - out).abs()
    # scores to about 30 * 8 * 4 = 960 in row 0 and 56 in row 2, as sums of 64 products: FP32's 2^-24 of their size, times 64 for
    # the sum, bounds the weights' relative error by 960 * 64 * 2^-24 = 2^-8 in row 0
    tol = 2.0 ** -8 * out.abs() + 2.0 ** -7 * size
    assert bool((err <= tol).all())
    b.kp[t[0, 3], 0, 5, 0] = float("inf")                       # an infinite key: an infinite score, NaN as exp(inf - inf)
    b.vp[t[1, 0], 0, 0, 7] = float("nan")                       # a NaN among the values stays in its component
    nwc.nwc_attend(b.call())
    torch.cuda.synchronize()
    up = b.q[0, :, 0] > 0
    assert bool(b.out[0][up].isnan().all()) and bool((~b.out[0][~up].isnan()).all())
    assert bool(b.out[1, :, 7].isnan().all()) and int(b.out[1].isnan().sum()) == 4
    assert not bool(b.out[2].isnan().any())


@pytest.mark.parametrize("covers", [0, 4000])
@pytest.mark.parametrize("hq,hk,d,page", [(32, 8, 128, 64), (16, 1, 64, 16), (5, 5, 96, 32), (8, 1, 256, 16), (10, 5, 192, 32)])
def test_attend_weights_of_16_bits(hq, hk, d, page, covers):
    # up to 16 columns a wavefront a weight is two BF16 values: the first leaves at most 2^-8 of it, the second 2^-8 of that
    _say("attend 16-bit weights %d %d %d %d %d" % (hq, hk, d, page, covers))
    groups = [(0, 4, 70), (6, 8, 33)] if 4 * hq // hk <= 64 else []
    b = _Batch([75, 90, 71, 104, 2, 3, 40, 35, 17, 64, 333], hq, hk, d, page, groups, seed=hq + d, covers=covers)
    nwc.nwc_attend(b.call())
    torch.cuda.synchronize()
    out, size = _ref_attend(b.kp, b.vp, b.table, b.lengths, b.q, b.scale)
    err = (b.out[:len(b.lengths)].double() - out).abs()
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -16 + 2.0 ** -10) * size
    assert bool((err <= tol).all()), "%g over its tolerance" % float((err - tol).max())


@pytest.mark.parametrize("covers", [0, 4000])
@pytest.mark.parametrize("hq,hk,d,page", SHAPES + [(20, 1, 128, 16), (32, 1, 64, 32)])
def test_attend_of_equal_values_is_the_value(hq, hk, d, page, covers):
    # the weights that the products take add up to the sum that they are divided by, to 2^-16 and FP32's 2^-24 a term
    # (1100 terms: 2^-13): far less than half a step of BF16, so what every position holds comes back as it is
    _say("attend equal values %d %d %d %d %d" % (hq, hk, d, page, covers))
    b = _Batch([600, 640, 555, 1100, 700, 600, 1, 33], hq, hk, d, page, [(0, 6, 550)], seed=hq * d, spread=3.0, covers=covers)
    value = _randn(torch.Generator(device="cuda").manual_seed(5), 1, hk, 1, d)
    b.vp.copy_(value.expand_as(b.vp))
    nwc.nwc_attend(b.call())
    torch.cuda.synchronize()
    want = value[0, :, 0].repeat_interleave(hq // hk, 0)
    assert torch.equal(b.out[:8], want.expand(8, hq, d))


@pytest.mark.parametrize("more", [0, 300])
def test_attend_strided_rows_and_far_pages(more):
    # queries inside a joint projection's rows, outputs inside a wider buffer, pages more than 2^32 elements apart
    d, hq, hk, page = 128, 8, 2, 16
    far = (1 << 32) + 8 * 1024
    room = torch.empty(2 * far + 2 * hk * page * d, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    kp, vp = (room[o:].as_strided((3, hk, page, d), (far, page * d, d, 1)) for o in (0, hk * page * d))
    kp.copy_(_randn(g, 3, hk, page, d))
    vp.copy_(_randn(g, 3, hk, page, d))
    x, wide = _randn(g, 2, (hq + 2 * hk) * d), torch.full((2, hq * d + 40), 7.0, dtype=torch.bfloat16, device="cuda")
    q, out = x[:, :hq * d].view(2, hq, d), wide[:, 8:8 + hq * d].view(2, hq, d)
    table, lengths = np.array([[2, 1] + [-1] * more, [0, 2] + [7] * more]), np.array([32, 21])
    cache = nwc.PagedCache(kp, vp)
    ws = torch.empty(nwc.nwc_attend_workspace_size(cache, 2, hq), dtype=torch.uint8, device="cuda")
    new = _randn(g, 1, 2 * hk * d)
    nwc.nwc_kv_append(nwc.KvAppend(cache, _i32(table), new[:, :hk * d].view(1, hk, d), new[:, hk * d:].view(1, hk, d), _i32([20]),
                                   rows=_i32([1])))
    nwc.nwc_attend(nwc.Attend(cache, _i32(table), _i32(lengths), q, out, ws))
    torch.cuda.synchronize()
    assert torch.equal(kp[2, :, 4], new[0, :hk * d].view(hk, d)) and torch.equal(vp[2, :, 4], new[0, hk * d:].view(hk, d))
    _check_attend(out, _ref_attend(kp, vp, table, lengths, q, d ** -0.5), "far pages")
    assert bool((wide[:, :8] == 7.0).all()) and bool((wide[:, 8 + hq * d:] == 7.0).all())


def test_attend_many_rows():
    rnd = np.random.default_rng(2)
    b = _Batch(rnd.integers(-1, 40, 4096), 4, 2, 64, 16, [(i * 32, i * 32 + 32, 8) for i in range(128)], seed=4)
    nwc.nwc_attend(b.call())
    torch.cuda.synchronize()
    b.check("4096 rows")


@pytest.mark.parametrize("covers", [0, 4000])
def test_decode_loop_in_a_graph(covers):
    """A prompt appended to two sequences, a shared copy for four continuations, then steps of append and attention
    as one captured graph whose positions and lengths move on the device; a second workspace user in between."""
    hq, hk, d, page, prompt, steps = 8, 2, 128, 16, 45, 6
    g = torch.Generator(device="cuda").manual_seed(11)
    freqs = _freqs(d)
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2))
    n_pages = 40
    kp, vp = (torch.full((n_pages, hk, page, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache = nwc.PagedCache(kp, vp)
    cols = -(-(prompt + steps) // page)
    table = np.random.default_rng(0).permutation(n_pages)[:4 * cols].reshape(4, cols)
    table[1:, :prompt // page] = table[0, :prompt // page]      # whole pages of the prompt are shared
    table = np.concatenate([table, np.full((4, -(-covers // page)), -1, np.int64)], 1)
    x = _randn(g, prompt, 2 * hk * d)
    rows, pos = _i32([0] * prompt), _i32(range(prompt))
    tab = _i32(table)
    nwc.nwc_kv_append(nwc.KvAppend(cache, tab, x[:, :hk * d].view(prompt, hk, d), x[:, hk * d:].view(prompt, hk, d), pos, rows=rows,
                                   k_weight=wk, freqs=freqs))
    tail = prompt % page                                        # the page that the prompt ends in: one copy each
    for r in range(1, 4):
        for p in (kp, vp):
            p[table[r, prompt // page], :, :tail] = p[table[0, prompt // page], :, :tail]
    xs = [_randn(g, 4, (hq + 2 * hk) * d) for _ in range(steps)]
    cur = torch.empty_like(xs[0])
    q, k, v = cur[:, :hq * d].view(4, hq, d), cur[:, hq * d:(hq + hk) * d].view(4, hk, d), cur[:, (hq + hk) * d:].view(4, hk, d)
    q_rot, out = torch.empty((4, hq, d), dtype=torch.bfloat16, device="cuda"), torch.empty((4, hq, d), dtype=torch.bfloat16, device="cuda")
    position, lengths = _i32([prompt] * 4), _i32([prompt + 1] * 4)
    ws = torch.empty(nwc.nwc_attend_workspace_size(cache, 4, hq, 1), dtype=torch.uint8, device="cuda")
    append = nwc.KvAppend(cache, tab, k, v, position, k_weight=wk, q=q, q_out=q_rot, q_weight=wq, freqs=freqs)
    attend = nwc.Attend(cache, tab, lengths, q_rot, out, ws, group_start=_i32([0, 4]), shared_len=_i32([prompt]))
    stream = torch.cuda.Stream()
    k_start, v_start = kp.clone(), vp.clone()
    cur.copy_(xs[0])
    torch.cuda.synchronize()

    def step():
        nwc.nwc_kv_append(append, stream=stream)
        nwc.nwc_attend(attend, stream=stream)

    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
        position.add_(1)
        lengths.add_(1)
    other = _Batch([70, 3], hq, hk, d, page, seed=1)
    other.ws = ws                                               # another caller of the same workspace, in order
    for replay in range(2):                                     # the second pass must repeat the first one's bits
        kp.copy_(k_start)
        vp.copy_(v_start)
        position.fill_(prompt)
        lengths.fill_(prompt + 1)
        outs = []
        for i in range(steps):
            cur.copy_(xs[i])
            torch.cuda.synchronize()
            with torch.cuda.stream(stream):
                graph.replay()
            torch.cuda.synchronize()
            outs.append(out.clone())
            qr, qs = _ref_heads(q, wq, _i32([prompt + i] * 4), freqs, "half")
            ref = _ref_attend(kp, vp, table, np.full(4, prompt + i + 1), q_rot, d ** -0.5)
            _check_attend(out, ref, "step %d" % i)
            _check_heads(q_rot, qr, qs, "queries of step %d" % i)
            nwc.nwc_attend(other.call())
            torch.cuda.synchronize()
        if replay:
            assert all(torch.equal(a, b) for a, b in zip(outs, first))
        first = outs
    other.check("the other caller")


@pytest.mark.parametrize("covers", [0, 5000])
def test_attend_graph_and_streams(covers):
    """Captured once, replayed with other lengths, queries and pages in the same buffers, against eager calls; two streams
    with a workspace each at once."""
    b = _Batch([300, 40, 511, 1], 16, 4, 128, 32, seed=9, covers=covers)
    lengths, table = _i32(b.lengths), _i32(b.table)
    call = nwc.Attend(b.cache, table, lengths, b.q, b.out[:4], b.ws, b.scale)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    nwc.nwc_attend(call, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        nwc.nwc_attend(call)                                    # the current stream: the one being captured
    torch.cuda.synchronize()
    for n, order in (([300, 40, 511, 1], [0, 1, 2, 3]), ([7, 40, 0, 1], [0, 1, 2, 3]), ([500, 33, 299, -1], [2, 1, 0, 3])):
        b.out.fill_(7.0)
        lengths.copy_(_i32(n))
        table.copy_(_i32(b.table[order]))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        n, live = np.array(n), torch.from_numpy(np.array(n) >= 0).cuda()
        out, size = _ref_attend(b.kp, b.vp, b.table[order], n, b.q, b.scale)
        _check_attend(b.out[:4][live], (out[live], size[live]), "replay")
        got = b.out.clone()
        nwc.nwc_attend(nwc.Attend(b.cache, _i32(b.table[order]), _i32(n), b.q, b.out[:4], b.ws, b.scale))
        torch.cuda.synchronize()
        assert torch.equal(got, b.out)
    other = _Batch([900, 77], 8, 2, 64, 16, seed=10, covers=covers)
    calls = [x.call() for x in (b, other)]
    streams = [torch.cuda.Stream() for _ in calls]
    for x in (b, other):
        x.out.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(calls, streams):
            nwc.nwc_attend(c, stream=s)
    torch.cuda.synchronize()
    b.check("first stream")
    other.check("second stream")


def test_calls_refuse_mixed_tensors():
    b = _Batch([5], 8, 2, 64, 16, seed=1)
    good = dict(cache=b.cache, table=_i32(b.table), lengths=_i32([5]), q=b.q, out=b.out[:1], ws=b.ws)
    for name, bad in (("q", b.q.float()), ("q", b.q[:, :, :32]), ("q", b.q.cpu()), ("out", b.out), ("lengths", _i32([5, 6])),
                      ("lengths", torch.tensor([5], device="cuda")), ("table", _i32(b.table).long()), ("ws", b.ws.cpu())):
        with pytest.raises(ValueError):
            nwc.Attend(**dict(good, **{name: bad}))
    with pytest.raises(ValueError):
        nwc.Attend(**good, group_start=_i32([0, 1]))
    with pytest.raises(nwc.NwcError):
        nwc.nwc_attend(nwc.Attend(**dict(good, ws=b.ws[:256])))
    with pytest.raises(nwc.NwcError):
        nwc.nwc_attend(nwc.Attend(**good, scale=0.0))
    with pytest.raises(ValueError):
        nwc.QkNormRope(b.q, None, _i32([0]), freqs=_freqs(32), style="thirds")
    with pytest.raises(nwc.NwcError):
        nwc.nwc_qk_norm_rope(nwc.QkNormRope(b.q, None, _i32([0]), freqs=_freqs(128)))   # more than the head has
