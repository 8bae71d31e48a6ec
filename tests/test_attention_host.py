"""The attention side on the host (no GPU): refusals of the C ABI before any
device work, and the binding's checks of tensors."""
import ctypes

import pytest
import torch

import decode_gemv_byte_amd as nwc

L = nwc._lib
A = 0x100000          # a 256-aligned fake device address, never used: every call here fails its checks


def _heads(src=A, dst=A, weight=None, ld_src=4096, ld_dst=4096, heads=32, reserved=0):
    return nwc.nwc_heads(src, dst, weight, ld_src, ld_dst, heads, reserved)


def _cache(k=A, v=A, n_pages=4, page_stride=8 * 64 * 128, kv_heads=8, head_dim=128, page_len=64, reserved=0):
    return nwc.nwc_cache(k, v, n_pages, page_stride, kv_heads, head_dim, page_len, reserved)


def _table(ids=A, ld=4, rows=2, cols=4):
    return nwc.nwc_page_table(ids, ld, rows, cols)


def _rope(freqs=A, dims=128, style=0):
    return nwc.nwc_rope(freqs, dims, style)


def _ref(x):
    return None if x is None else ctypes.byref(x)


def _norm_rope(q=None, k=None, tokens=2, d=128, eps=1e-6, rope=None, positions=A):
    return L.nwc_qk_norm_rope(_ref(q), _ref(k), tokens, d, eps, _ref(rope), positions, None)


def test_norm_rope_refusals():
    q = _heads()
    assert _norm_rope() == nwc.NWC_ERR_INVALID_ARG                                     # neither
    assert _norm_rope(q, tokens=0) == nwc.NWC_ERR_INVALID_ARG
    assert _norm_rope(q, positions=None) == nwc.NWC_ERR_INVALID_ARG
    assert _norm_rope(q, positions=A + 2) == nwc.NWC_ERR_ALIGNMENT
    for eps in (-1e-6, float("nan"), float("inf")):
        assert _norm_rope(q, eps=eps) == nwc.NWC_ERR_INVALID_ARG
    assert _norm_rope(q, d=0) == nwc.NWC_ERR_INVALID_ARG
    for d in (4, 100, 264, 512):
        assert _norm_rope(q, d=d) == nwc.NWC_ERR_UNSUPPORTED
    for bad, want in ((dict(src=None), nwc.NWC_ERR_INVALID_ARG), (dict(dst=None), nwc.NWC_ERR_INVALID_ARG),
                      (dict(heads=0), nwc.NWC_ERR_INVALID_ARG), (dict(heads=70000, ld_src=1 << 30, ld_dst=1 << 30), nwc.NWC_ERR_INVALID_ARG),
                      (dict(ld_src=4088), nwc.NWC_ERR_INVALID_ARG), (dict(ld_dst=4088), nwc.NWC_ERR_INVALID_ARG),
                      (dict(ld_src=1 << 50), nwc.NWC_ERR_INVALID_ARG), (dict(reserved=1), nwc.NWC_ERR_INVALID_ARG),
                      (dict(ld_dst=4104), nwc.NWC_ERR_INVALID_ARG),                    # in place with another stride
                      (dict(src=A + 2), nwc.NWC_ERR_ALIGNMENT), (dict(dst=A + 8), nwc.NWC_ERR_ALIGNMENT),
                      (dict(weight=A + 4), nwc.NWC_ERR_ALIGNMENT), (dict(ld_src=4100), nwc.NWC_ERR_ALIGNMENT),
                      (dict(dst=A + 4096, ld_dst=4100), nwc.NWC_ERR_ALIGNMENT)):
        assert _norm_rope(_heads(**bad)) == want, bad
        assert _norm_rope(None, _heads(**bad)) == want, bad
    for bad, want in ((dict(freqs=None), nwc.NWC_ERR_INVALID_ARG), (dict(dims=144), nwc.NWC_ERR_INVALID_ARG),
                      (dict(style=2), nwc.NWC_ERR_INVALID_ARG), (dict(dims=20), nwc.NWC_ERR_UNSUPPORTED),
                      (dict(dims=1), nwc.NWC_ERR_UNSUPPORTED), (dict(freqs=A + 2), nwc.NWC_ERR_ALIGNMENT)):
        assert _norm_rope(q, rope=_rope(**bad)) == want, bad


def _append(cache="", table="", k="", v=A, ld_v=1024, q=None, tokens=2, eps=1e-6, rope=None, positions=A, rows=None):
    cache = _cache() if cache == "" else cache
    table = _table() if table == "" else table
    k = _heads(heads=8, ld_src=1024) if k == "" else k
    return L.nwc_kv_append(_ref(cache), _ref(table), _ref(k), v, ld_v, _ref(q), tokens, eps, _ref(rope), positions, rows, None)


CACHE_BAD = ((dict(k=None), nwc.NWC_ERR_INVALID_ARG), (dict(v=None), nwc.NWC_ERR_INVALID_ARG),
             (dict(n_pages=0), nwc.NWC_ERR_INVALID_ARG), (dict(n_pages=1 << 31), nwc.NWC_ERR_INVALID_ARG),
             (dict(page_stride=8 * 64 * 128 - 8), nwc.NWC_ERR_INVALID_ARG), (dict(page_stride=1 << 50), nwc.NWC_ERR_INVALID_ARG),
             (dict(kv_heads=0), nwc.NWC_ERR_INVALID_ARG), (dict(page_len=0), nwc.NWC_ERR_INVALID_ARG),
             (dict(reserved=3), nwc.NWC_ERR_INVALID_ARG), (dict(page_len=8), nwc.NWC_ERR_UNSUPPORTED),
             (dict(page_len=48), nwc.NWC_ERR_UNSUPPORTED), (dict(page_len=2048, page_stride=1 << 30), nwc.NWC_ERR_UNSUPPORTED),
             (dict(k=A + 8), nwc.NWC_ERR_ALIGNMENT), (dict(v=A + 2), nwc.NWC_ERR_ALIGNMENT),
             (dict(page_stride=8 * 64 * 128 + 4), nwc.NWC_ERR_ALIGNMENT))
TABLE_BAD = ((dict(ids=None), nwc.NWC_ERR_INVALID_ARG), (dict(rows=0), nwc.NWC_ERR_INVALID_ARG),
             (dict(cols=0), nwc.NWC_ERR_INVALID_ARG), (dict(ld=3), nwc.NWC_ERR_INVALID_ARG),
             (dict(ids=A + 1), nwc.NWC_ERR_ALIGNMENT))


def test_append_refusals():
    for name in ("cache", "table", "k", "v", "positions"):
        assert _append(**{name: None}) == nwc.NWC_ERR_INVALID_ARG, name
    assert _append(tokens=0) == nwc.NWC_ERR_INVALID_ARG
    assert _append(tokens=3) == nwc.NWC_ERR_INVALID_ARG                                # token t is row t, two rows
    assert _append(eps=-1.0) == nwc.NWC_ERR_INVALID_ARG
    assert _append(ld_v=1016) == nwc.NWC_ERR_INVALID_ARG
    assert _append(ld_v=1028) == nwc.NWC_ERR_ALIGNMENT
    assert _append(v=A + 2) == nwc.NWC_ERR_ALIGNMENT
    assert _append(positions=A + 1) == nwc.NWC_ERR_ALIGNMENT
    assert _append(rows=A + 2) == nwc.NWC_ERR_ALIGNMENT
    assert _append(k=_heads(heads=4)) == nwc.NWC_ERR_INVALID_ARG                       # the cache has 8 heads
    assert _append(q=_heads(dst=None)) == nwc.NWC_ERR_INVALID_ARG
    assert _append(rope=_rope(dims=20)) == nwc.NWC_ERR_UNSUPPORTED
    assert _append(cache=_cache(head_dim=0)) == nwc.NWC_ERR_INVALID_ARG
    assert _append(cache=_cache(head_dim=100)) == nwc.NWC_ERR_UNSUPPORTED
    for bad, want in CACHE_BAD:
        assert _append(cache=_cache(**bad)) == want, bad
    for bad, want in TABLE_BAD:
        assert _append(table=_table(**bad)) == want, bad


def _attend(cache="", table="", groups=None, lengths=A, q=A, ldq=4096, hq=32, scale=0.1, out=A, ldo=4096, ws=A, n=1 << 40):
    cache = _cache() if cache == "" else cache
    table = _table() if table == "" else table
    return L.nwc_attend(_ref(cache), _ref(table), _ref(groups), lengths, q, ldq, hq, scale, out, ldo, ws, n, None)


def test_attend_refusals():
    for name in ("cache", "table", "lengths", "q", "out", "ws"):
        assert _attend(**{name: None}) == nwc.NWC_ERR_INVALID_ARG, name
    for scale in (0.0, -0.1, float("nan"), float("inf")):
        assert _attend(scale=scale) == nwc.NWC_ERR_INVALID_ARG
    assert _attend(hq=0) == nwc.NWC_ERR_INVALID_ARG
    assert _attend(hq=30) == nwc.NWC_ERR_INVALID_ARG                                   # no multiple of 8
    assert _attend(hq=8 * 65, ldq=1 << 20, ldo=1 << 20) == nwc.NWC_ERR_UNSUPPORTED
    for name in ("ldq", "ldo"):
        assert _attend(**{name: 4088}) == nwc.NWC_ERR_INVALID_ARG
        assert _attend(**{name: 4100}) == nwc.NWC_ERR_ALIGNMENT
        assert _attend(**{name: 1 << 50}) == nwc.NWC_ERR_INVALID_ARG
    for name in ("q", "out", "ws"):
        assert _attend(**{name: A + 8}) == nwc.NWC_ERR_ALIGNMENT
    assert _attend(ws=A + 128) == nwc.NWC_ERR_ALIGNMENT
    assert _attend(lengths=A + 2) == nwc.NWC_ERR_ALIGNMENT
    for d in (32, 80, 112, 160):
        assert _attend(cache=_cache(head_dim=d, page_stride=1 << 20)) == nwc.NWC_ERR_UNSUPPORTED
    assert _attend(table=_table(rows=4097)) == nwc.NWC_ERR_UNSUPPORTED
    assert _attend(table=_table(cols=65537, ld=65537)) == nwc.NWC_ERR_UNSUPPORTED      # 64 * 65537 > 2^22 positions
    g = nwc.nwc_groups
    assert _attend(groups=g(None, A, 1, 0)) == nwc.NWC_ERR_INVALID_ARG
    assert _attend(groups=g(A, None, 1, 0)) == nwc.NWC_ERR_INVALID_ARG
    assert _attend(groups=g(A, A, 1, 5)) == nwc.NWC_ERR_INVALID_ARG
    assert _attend(groups=g(A, A, 513, 0)) == nwc.NWC_ERR_UNSUPPORTED
    assert _attend(groups=g(A + 2, A, 1, 0)) == nwc.NWC_ERR_ALIGNMENT
    assert _attend(groups=g(A, A + 1, 1, 0)) == nwc.NWC_ERR_ALIGNMENT
    for bad, want in CACHE_BAD:
        assert _attend(cache=_cache(**bad)) == want, bad
    for bad, want in TABLE_BAD:
        assert _attend(table=_table(**bad)) == want, bad
    size = ctypes.c_size_t()
    assert L.nwc_attend_workspace_size(_ref(_cache()), 2, 32, 0, ctypes.byref(size)) == nwc.NWC_OK
    assert size.value % 256 == 0 and size.value > 0
    assert _attend(n=size.value - 1) == nwc.NWC_ERR_BUFFER_TOO_SMALL
    assert L.nwc_attend_workspace_size(_ref(_cache()), 2, 32, 0, None) == nwc.NWC_ERR_INVALID_ARG
    assert L.nwc_attend_workspace_size(None, 2, 32, 0, ctypes.byref(size)) == nwc.NWC_ERR_INVALID_ARG
    assert L.nwc_attend_workspace_size(_ref(_cache()), 0, 32, 0, ctypes.byref(size)) == nwc.NWC_ERR_INVALID_ARG
    assert L.nwc_attend_workspace_size(_ref(_cache()), 2, 31, 0, ctypes.byref(size)) == nwc.NWC_ERR_INVALID_ARG
    assert L.nwc_attend_workspace_size(_ref(_cache(head_dim=80)), 2, 32, 0, ctypes.byref(size)) == nwc.NWC_ERR_UNSUPPORTED
    before = size.value
    assert L.nwc_attend_workspace_size(_ref(_cache()), 2, 32, 2, ctypes.byref(size)) == nwc.NWC_OK and size.value >= before


def test_attend_refuses_output_over_queries_and_oversized_launches():
    assert _attend(q=A, out=A) == nwc.NWC_ERR_INVALID_ARG
    # a launch holds fewer than 2^32 threads: rows times query heads up to 2^22
    size = ctypes.c_size_t()
    many = _cache(kv_heads=1024, page_stride=1024 * 64 * 128)
    assert L.nwc_attend_workspace_size(_ref(many), 4096, 1024, 0, ctypes.byref(size)) == nwc.NWC_OK
    assert L.nwc_attend_workspace_size(_ref(many), 4096, 2048, 0, ctypes.byref(size)) == nwc.NWC_ERR_UNSUPPORTED
    assert _attend(cache=many, table=_table(rows=4096), hq=2048, ldq=1 << 20, ldo=1 << 20, out=1 << 40) == nwc.NWC_ERR_UNSUPPORTED


def test_binding_refuses_host_tensors_and_odd_layouts():
    pages = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16)
    cache = nwc.PagedCache(pages, pages.clone())
    assert (cache.struct.n_pages, cache.struct.kv_heads, cache.struct.page_len, cache.struct.head_dim) == (2, 1, 16, 64)
    assert cache.struct.page_stride == 16 * 64
    wide = torch.zeros((2, 2, 1, 16, 64), dtype=torch.bfloat16)
    assert nwc.PagedCache(wide[:, 0], wide[:, 1]).struct.page_stride == 2 * 16 * 64
    with pytest.raises(ValueError):
        nwc.PagedCache(pages, pages[:1])                       # another shape
    with pytest.raises(ValueError):
        nwc.PagedCache(pages.transpose(1, 2), pages.transpose(1, 2))
    with pytest.raises(ValueError):
        nwc.PagedCache(wide[:, 0], pages)                      # pages another distance apart
    q = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    pos = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        nwc.QkNormRope(q, None, pos)                           # on the host
    with pytest.raises(ValueError):
        nwc.QkNormRope(None, None, pos)
    with pytest.raises(ValueError):
        nwc.KvAppend(cache, torch.zeros((1, 2), dtype=torch.int32), q, q, pos)
    with pytest.raises(ValueError):
        nwc.Attend(cache, torch.zeros((3, 2), dtype=torch.int32), pos, q, q, torch.zeros(8, dtype=torch.uint8))


def test_paged_cache_takes_any_stride_of_one_head():
    # a head's share of a joint allocation for several: the stride of a dimension of one entry means nothing
    joint = torch.zeros((3, 4, 16, 64), dtype=torch.bfloat16)
    cache = nwc.PagedCache(joint[:, :1], joint[:, 2:3])
    assert (cache.struct.kv_heads, cache.struct.page_stride) == (1, 4 * 16 * 64)
    assert cache.struct.v - cache.struct.k == 2 * 16 * 64 * 2
    moved = joint.as_strided((3, 1, 16, 64), (4 * 16 * 64, 7, 64, 1))
    assert nwc.PagedCache(moved, moved).struct.page_stride == 4 * 16 * 64
    with pytest.raises(ValueError):
        nwc.PagedCache(joint[:, ::2], joint[:, ::2])           # two heads, not side by side
    with pytest.raises(ValueError):
        nwc.PagedCache(joint[:, :, ::2], joint[:, :, ::2])     # every second slot
    with pytest.raises(ValueError):
        nwc.PagedCache(joint[..., ::2], joint[..., ::2])
