"""Chunk attention, the residual norm and token log probabilities on the host (no
GPU): refusals of the C ABI before any device work, and the binding's checks of
tensors."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import decode_gemv_byte_amd as nwc
from test_attention_host import A, CACHE_BAD, TABLE_BAD, _cache, _ref, _table

L = nwc._lib
INVALID, SMALL, UNSUPPORTED, ALIGN = (nwc.NWC_ERR_INVALID_ARG, nwc.NWC_ERR_BUFFER_TOO_SMALL, nwc.NWC_ERR_UNSUPPORTED,
                                      nwc.NWC_ERR_ALIGNMENT)


def _chunk(cache="", table="", start=A, lengths=A, q=A, ldq=4096, tokens=7, hq=32, scale=0.1, out=2 * A, ldo=4096, ws=A, n=1 << 40):
    cache = _cache() if cache == "" else cache
    table = _table() if table == "" else table
    return L.nwc_attend_chunk(_ref(cache), _ref(table), start, lengths, q, ldq, tokens, hq, scale, out, ldo, ws, n, None)


def test_chunk_refusals():
    for name in ("cache", "table", "start", "lengths", "q", "out", "ws"):
        assert _chunk(**{name: None}) == INVALID, name
    for scale in (0.0, -0.1, float("nan"), float("inf"), 3e38):
        assert _chunk(scale=scale) == INVALID
    assert _chunk(tokens=0) == INVALID
    assert _chunk(hq=0) == INVALID
    assert _chunk(hq=30) == INVALID                                                    # no multiple of 8
    assert _chunk(hq=8 * 65, ldq=1 << 20, ldo=1 << 20) == UNSUPPORTED
    assert _chunk(tokens=(1 << 22) + 1) == UNSUPPORTED
    assert _chunk(q=A, out=A) == INVALID
    for name in ("ldq", "ldo"):
        assert _chunk(**{name: 4088}) == INVALID
        assert _chunk(**{name: 4100}) == ALIGN
        assert _chunk(**{name: 1 << 50}) == INVALID
    for name in ("q", "out", "ws"):
        assert _chunk(**{name: A + 8}) == ALIGN
    assert _chunk(ws=A + 128) == ALIGN
    assert _chunk(lengths=A + 2) == ALIGN and _chunk(start=A + 1) == ALIGN
    for d in (32, 80, 112, 160):
        assert _chunk(cache=_cache(head_dim=d, page_stride=1 << 20)) == UNSUPPORTED
    assert _chunk(table=_table(rows=4097)) == UNSUPPORTED
    assert _chunk(table=_table(cols=65537, ld=65537)) == UNSUPPORTED                   # 64 * 65537 > 2^22 positions
    for bad, want in CACHE_BAD:
        assert _chunk(cache=_cache(**bad)) == want, bad
    for bad, want in TABLE_BAD:
        assert _chunk(table=_table(**bad)) == want, bad
    size = ctypes.c_size_t()
    fn = L.nwc_attend_chunk_workspace_size
    assert fn(_ref(_cache()), 2, 7, 32, ctypes.byref(size)) == nwc.NWC_OK and size.value % 256 == 0 and size.value > 0
    assert _chunk(n=size.value - 1) == SMALL
    assert fn(_ref(_cache()), 2, 7, 32, None) == INVALID and fn(None, 2, 7, 32, ctypes.byref(size)) == INVALID
    assert fn(_ref(_cache()), 0, 7, 32, ctypes.byref(size)) == INVALID and fn(_ref(_cache()), 2, 0, 32, ctypes.byref(size)) == INVALID
    assert fn(_ref(_cache()), 2, 7, 31, ctypes.byref(size)) == INVALID
    assert fn(_ref(_cache(head_dim=80)), 2, 7, 32, ctypes.byref(size)) == UNSUPPORTED
    # every number of query heads a key-value head has whole tokens in an item, and room for them
    for ratio in range(1, 65):
        assert fn(_ref(_cache()), 4096, 1 << 22, 8 * ratio, ctypes.byref(size)) == nwc.NWC_OK
        assert size.value >= 2 * 256 * (128 // ratio * ratio) * 128 * 4


def _residual(x=A, x_out=2 * A, y=3 * A, y_weight=None, gate=None, weight=A, out=4 * A, ld_x=64, ld_x_out=64, ld_y=64, ld_gate=0,
              ld_out=64, scale=1.0, eps=1e-6, x_type=0, reserved=0, tokens=3, cols=64):
    a = nwc.nwc_residual(x, x_out, y, y_weight, gate, weight, out, ld_x, ld_x_out, ld_y, ld_gate, ld_out, scale, eps, x_type, reserved)
    return L.nwc_residual_norm(ctypes.byref(a), tokens, cols, None)


def test_residual_refusals():
    assert L.nwc_residual_norm(None, 1, 64, None) == INVALID
    for bad in (dict(x=None), dict(tokens=0), dict(cols=0), dict(reserved=1), dict(x_type=2), dict(eps=-1.0), dict(eps=float("nan")),
                dict(scale=float("inf")), dict(weight=None), dict(out=None), dict(out=None, weight=None, x_out=None),
                dict(y=None), dict(y=None, x_out=None, gate=A), dict(y=None, x_out=None, y_weight=A),
                dict(ld_x=56), dict(ld_x_out=56), dict(ld_y=56), dict(ld_out=56), dict(gate=A, ld_gate=56), dict(ld_x=1 << 50),
                dict(x_out=A, ld_x_out=72), dict(out=2 * A), dict(out=3 * A, ld_out=72), dict(out=A, x_out=None, ld_out=72),
                dict(out=A, x_out=None, x_type=1), dict(x_out=3 * A), dict(gate=5 * A, out=5 * A), dict(gate=5 * A, x_out=5 * A),
                dict(weight=4 * A), dict(weight=2 * A), dict(y_weight=2 * A), dict(y_weight=4 * A)):
        assert _residual(**bad) == INVALID, bad
    for cols in (4, 100, 32776, 65536):
        assert _residual(cols=cols, ld_x=1 << 20, ld_x_out=1 << 20, ld_y=1 << 20, ld_out=1 << 20) == UNSUPPORTED
    for name in ("x", "x_out", "y", "y_weight", "gate", "weight", "out"):
        assert _residual(**{name: 7 * A + 8}) == ALIGN, name
    for bad in (dict(ld_x=68), dict(ld_x_out=68), dict(ld_y=68), dict(ld_out=68), dict(gate=A, ld_gate=68)):
        assert _residual(**bad) == ALIGN, bad


def _logprobs(logits=A, ld=1008, type=0, rows=3, vocab=1001, scale=1.0, targets=A, n=2, logprobs=A, entropy=A, k=5, ids=A, top=A,
              ws=A, size=1 << 40):
    return L.nwc_token_logprobs(logits, ld, type, rows, vocab, scale, targets, n, logprobs, entropy, k, ids, top, ws, size, None)


def test_logprobs_refusals():
    for bad in (dict(logits=None), dict(ws=None), dict(type=2), dict(rows=0), dict(vocab=0), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(targets=None), dict(logprobs=None), dict(n=0),
                dict(ids=None), dict(top=None), dict(k=0), dict(ld=1000), dict(ld=1 << 50),
                dict(vocab=4, k=5), dict(targets=None, n=0, logprobs=None, entropy=None, k=0, ids=None, top=None)):
        assert _logprobs(**bad) == INVALID, bad
    for bad in (dict(k=65), dict(n=65537), dict(rows=(1 << 22) + 1), dict(vocab=1 << 31, ld=1 << 32)):
        assert _logprobs(**bad) == UNSUPPORTED, bad
    for bad in (dict(logits=A + 8), dict(ld=1004), dict(ld=1010, type=1), dict(targets=A + 2), dict(logprobs=A + 1), dict(entropy=A + 2),
                dict(ids=A + 2), dict(top=A + 2), dict(ws=A + 128)):
        assert _logprobs(**bad) == ALIGN, bad
    size = ctypes.c_size_t()
    fn = L.nwc_token_logprobs_workspace_size
    assert fn(3, 128256, 5, None) == INVALID and fn(0, 128256, 5, ctypes.byref(size)) == INVALID
    assert fn(3, 128256, 65, ctypes.byref(size)) == UNSUPPORTED
    assert fn(3, 128256, 5, ctypes.byref(size)) == nwc.NWC_OK and size.value % 256 == 0
    assert _logprobs(vocab=128256, ld=128256, size=size.value - 1) == SMALL


def test_binding_refuses_host_tensors_and_odd_calls():
    bf = torch.zeros((2, 64), dtype=torch.bfloat16)
    one = torch.zeros(64, dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError):
        nwc.ResidualNorm(bf, bf, out=bf, weight=one)                        # on the host
    with pytest.raises(ValueError):
        nwc.TokenLogprobs(bf, ws, entropy=torch.zeros(2))
    pages = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16)
    cache = nwc.PagedCache(pages, pages.clone())
    i = torch.zeros((1, 2), dtype=torch.int32)
    q = torch.zeros((2, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nwc.AttendChunk(cache, i, i[0], i[0, :1], q, q.clone(), ws)


def _kernels(tmp_path):
    """The kernels' metadata of every code object in the built library, by name."""
    import yaml
    objcopy, bundler, readelf = (os.path.join("/opt/rocm/llvm/bin", t) for t in ("llvm-objcopy", "clang-offload-bundler", "llvm-readelf"))
    if not all(os.path.exists(t) for t in (objcopy, bundler, readelf)):
        pytest.skip("ROCm LLVM tools not found")
    lib, fat, one, co = (str(tmp_path / n) for n in ("lib.so", "fat.bin", "one.bin", "co.o"))
    shutil.copy(nwc.LIB_PATH, lib)
    subprocess.run([objcopy, "--dump-section", ".hip_fatbin=" + fat, lib, str(tmp_path / "out.so")], check=True, capture_output=True)
    with open(fat, "rb") as f:
        parts = f.read().split(b"__CLANG_OFFLOAD_BUNDLE__")[1:]   # one of each source
    found = {}
    for part in parts:
        with open(one, "wb") as f:
            f.write(b"__CLANG_OFFLOAD_BUNDLE__" + part)
        subprocess.run([bundler, "--unbundle", "--type=o", "--input=" + one, "--targets=hipv4-amdgcn-amd-amdhsa--gfx950",
                        "--output=" + co], check=True, capture_output=True)
        notes = subprocess.run([readelf, "--notes", co], check=True, capture_output=True, text=True).stdout
        text = notes[notes.index("---"):]
        meta = yaml.safe_load(text[text.index("\n") + 1:text.index("\n...")])
        found.update({k[".name"]: k for k in meta["amdhsa.kernels"]})
    return found


def test_chunk_kernels_spill_nothing(tmp_path):
    # a register that is stored to memory where a branch has some lanes off comes back wrong for them, an address among
    # them: these kernels, near the most registers there are, keep all of theirs
    kernels = _kernels(tmp_path)
    ours = [k for n, k in kernels.items() if "k_chunk" in n or "k_logprobs" in n or "k_residual" in n]
    assert sum("k_chunk" in k[".name"] for k in ours) == 11 and sum("k_logprobs" in k[".name"] for k in ours) == 4
    for k in ours:
        assert k[".vgpr_spill_count"] == 0 and k[".private_segment_fixed_size"] == 0, k[".name"]


def test_a_workspace_for_more_serves_less():
    size = ctypes.c_size_t()

    def chunk(rows, tokens, ratio, hkv, d):
        c = _cache(head_dim=d, kv_heads=hkv, page_stride=hkv * d * 1024)
        assert L.nwc_attend_chunk_workspace_size(_ref(c), rows, tokens, ratio * hkv, ctypes.byref(size)) == nwc.NWC_OK
        return size.value
    for d in (64, 96, 128, 192, 256):
        for ratio, hkv in ((1, 8), (4, 8), (7, 4), (64, 1)):
            last = 0
            for tokens in list(range(1, 300)) + [500, 1000, 4096, 70000]:
                sizes = {chunk(rows, tokens, ratio, hkv, d) for rows in (1, 2, 5, 33, 700)}
                assert len(sizes) == 1 and sizes.pop() >= last, (d, ratio, tokens)
                last = chunk(1, tokens, ratio, hkv, d)

    def logprobs(rows, vocab, k):
        assert L.nwc_token_logprobs_workspace_size(rows, vocab, k, ctypes.byref(size)) == nwc.NWC_OK
        return size.value
    for vocab in (100, 4096, 4097, 32003, 128256, 1 << 20):
        for k in (0, 1, 20, 64):
            sizes = [logprobs(rows, vocab, k) for rows in list(range(1, 600)) + [1024, 4096]]
            assert sizes == sorted(sizes), (vocab, k)
            assert all(logprobs(rows, vocab, k) <= logprobs(rows, vocab + 5000, k) for rows in (1, 7, 300, 600))
