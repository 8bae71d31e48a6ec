"""The residual stream with the norms around a block, and token log probabilities,
on the GPU against plain 64-bit computations.

Tolerances, from the roundings:
 * BF16 results: half a step, 2^-8 of the value.  FP32 arithmetic before it: the sum
   x + scale gate u has a few roundings of 2^-24 of its terms, and each norm's sum of
   squares at most 8 + 8 + 16 additions in a row: 2^-17 of the terms' size covers it.
 * FP32 sums: 2^-17 of the normed part, and 2^-22 of the terms without a norm (three
   products and the sum).
 * log probabilities: (x - m) c is off by three roundings of itself (2^-22), a weight by
   that and the hardware's exp2 (2^-22 relative), sums by at most V / 4096 + 64
   additions in a row: 2^-24 (V / 4096 + 64) + 2^-21 ((m - x) scale + H + 1), H the
   entropy, which bounds the mean of (m - x) scale.  The entropy: the same with the second
   moment of (m - x) scale, 2^-24 (V / 4096 + 64) (1 + H) + 2^-21 (H + M2 + 1).
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


# ------------------------------------------------------ the residual stream ---

def _ref_residual(x, y, y_weight, gate, scale, weight, eps=EPS):
    """(sum, normed, size of the sum's terms) in 64 bits."""
    def normed(v, w):
        return v / (v.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    x = x.double()
    u = torch.zeros_like(x)
    if y is not None:
        u = y.double()
        if y_weight is not None:
            u = normed(u, y_weight)
        if gate is not None:
            u = u * gate.double()
        u = u * scale
    s = x + u
    return s, None if weight is None else normed(s, weight), x.abs() + u.abs()


def _check_residual(ref, x_out, out, weight, what, after):
    s, n, size = ref
    if x_out is not None:
        tol = (2.0 ** -17 if after else 2.0 ** -22) * size
        if x_out.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * s.abs()
        err = (x_out.double() - s).abs()
        assert bool((err <= tol).all()), "%s: sum %g over" % (what, float((err - tol).max()))
    if out is not None:
        r = 1 / (s.square().mean(-1, keepdim=True) + EPS).sqrt()
        tol = 2.0 ** -8 * n.abs() + 2.0 ** -16 * size * r * weight.double().abs()
        err = (out.double() - n).abs()
        assert bool((err <= tol).all()), "%s: normed %g over" % (what, float((err - tol).max()))


COLS = [(1, 8), (1, 4096), (3, 504), (5, 512), (2, 520), (37, 2560), (1, 8192), (2, 16384), (3, 32768), (1, 30000), (1030, 64),
        (1100, 1000), (1024, 2048), (1025, 4096), (1040, 4104), (1200, 8192), (1024, 16392), (2000, 520), (7, 12296)]


@pytest.mark.parametrize("tokens,cols", COLS)
@pytest.mark.parametrize("f32", [False, True])
def test_residual(tokens, cols, f32):
    g = torch.Generator(device="cuda").manual_seed(tokens + cols)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    x = (3 * rnd(tokens, cols + 16)).to(torch.float32 if f32 else torch.bfloat16)[:, :cols]
    y = rnd(tokens, cols + 8).to(torch.bfloat16)[:, :cols]
    w, yw, gv = ((1 + 0.3 * rnd(cols)).to(torch.bfloat16) for _ in range(3))
    gt = rnd(tokens, cols).to(torch.bfloat16)
    for after, gate, scale, before in ((None, None, 1.0, w), (yw, None, 1.0, w), (yw, gt, 0.22, w), (None, gv, -1.5, w), (yw, gv, 0.5, None)):
        what = "%d x %d %s after %s gate %s before %s" % (tokens, cols, "f32" if f32 else "bf16", after is not None,
                                                          None if gate is None else gate.dim(), before is not None)
        _say(what)
        wide = torch.full((tokens, cols + 24), 7.0, dtype=x.dtype, device="cuda")
        x_out = wide[:, :cols]
        out = torch.full((tokens, cols), 7.0, dtype=torch.bfloat16, device="cuda") if before is not None else None
        nwc.nwc_residual_norm(nwc.ResidualNorm(x, y, x_out=x_out, out=out, weight=before, y_weight=after, gate=gate, scale=scale,
                                               eps=EPS))
        torch.cuda.synchronize()
        ref = _ref_residual(x, y, after, gate, scale, before)
        _check_residual(ref, x_out, out, before, what, after is not None)
        assert bool((wide[:, cols:] == 7.0).all())
        # in place, the normed over the block's output, the same bits
        x2, y2 = x.clone(), y.clone()
        nwc.nwc_residual_norm(nwc.ResidualNorm(x2, y2, out=y2 if before is not None else None, weight=before, y_weight=after,
                                               gate=gate, scale=scale, eps=EPS))
        torch.cuda.synchronize()
        assert torch.equal(x2, x_out)
        if before is not None:
            assert torch.equal(y2, out)
    # the norm alone, and the normed sum without the sum
    out = torch.empty((tokens, cols), dtype=torch.bfloat16, device="cuda")
    nwc.nwc_residual_norm(nwc.ResidualNorm(x, out=out, weight=w, eps=EPS))
    before = x.clone()
    out2 = torch.empty_like(out)
    nwc.nwc_residual_norm(nwc.ResidualNorm(x, y, out=out2, weight=w, eps=EPS, keep=False))
    torch.cuda.synchronize()
    assert torch.equal(x, before)
    _check_residual(_ref_residual(x, None, None, None, 1.0, w), None, out, w, "norm alone", False)
    _check_residual(_ref_residual(x, y, None, None, 1.0, w), None, out2, w, "sum not kept", False)


def test_residual_special_values():
    cols = 1000
    x = torch.ones((7, cols), device="cuda")
    y = torch.zeros((7, cols), dtype=torch.bfloat16, device="cuda")
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    x[3] *= 2.0 ** 100
    x[4] *= 2.0 ** -120
    y[5, 7] = float("nan")
    y[6] = 2.0 ** 120
    one = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    out = torch.empty((7, cols), dtype=torch.bfloat16, device="cuda")
    x_out = torch.empty_like(x)
    nwc.nwc_residual_norm(nwc.ResidualNorm(x, y, x_out=x_out, out=out, weight=one, eps=0.0))
    torch.cuda.synchronize()
    assert bool(out[0].isnan().all())                          # zeros, no eps
    assert bool(out[1].isnan().all()) and bool(out[2].isnan().any()) and bool(out[5].isnan().all())
    for r in (3, 4, 6):
        assert torch.equal(out[r], one), r                     # a direction, whatever its size
    assert torch.equal(x_out[6], torch.full((cols,), 2.0 ** 120, device="cuda"))
    assert int(x_out[5].isnan().sum()) == 1 and int(x_out[1].isnan().sum()) == 1
    # the norm after a block: its rows of any size too, and zeros with eps add nothing
    y[6] = 2.0 ** 120
    y[5] = 2.0 ** -120
    y[4] = 0
    x.fill_(1.0)
    nwc.nwc_residual_norm(nwc.ResidualNorm(x[:, :], y, x_out=x_out, y_weight=one, eps=1e-30))
    torch.cuda.synchronize()
    assert torch.equal(x_out[6], torch.full((cols,), 2.0, device="cuda"))
    assert torch.equal(x_out[4], torch.ones(cols, device="cuda"))
    want = 1 + 2.0 ** -120 / (2.0 ** -240 + 1e-30) ** 0.5
    assert float((x_out[5] - want).abs().max()) <= 2.0 ** -22


# ------------------------------------------------------- log probabilities ---

def _ref_logprobs(x, scale):
    x = x.double()
    return torch.log_softmax(x * scale, -1)


def _check_logprobs(x, scale, targets, lp, ent, ids, top, what):
    V = x.shape[1]
    x = x.double()
    ref = torch.log_softmax(x * scale, -1)
    p = ref.exp()
    t = ((x.amax(-1, keepdim=True) - x) * scale).clamp(max=1e30)
    h = -(torch.where(p > 0, p * ref, 0.0)).sum(-1)
    m2 = torch.where(p > 0, p * t * t, 0.0).sum(-1)
    base = 2.0 ** -24 * (V / 4096 + 64)
    if targets is not None:
        idx = targets.long()
        ok = (idx >= 0) & (idx < V)
        safe = idx.clamp(0, V - 1)
        want = ref.gather(1, safe)
        tol = base + 2.0 ** -21 * (t.gather(1, safe) + h[:, None] + 1)
        same = (lp.double() == want) | ((lp.double() - want).abs() <= tol)
        assert bool((same | ~ok).all()), "%s: log probability off by %g" % (what, float((lp.double() - want).abs()[ok].max()))
        assert bool((lp[~ok] == 7.0).all()), "%s: no token, yet written" % what
    if ent is not None:
        err = (ent.double() - h).abs()
        assert bool((err <= base * (1 + h) + 2.0 ** -21 * (h + m2 + 1)).all()), "%s: entropy off by %g" % (what, float(err.max()))
    if ids is not None:
        k = ids.shape[1]
        order = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :k]
        assert torch.equal(ids.long(), order), "%s: top ids" % what
        want = ref.gather(1, order)
        tol = base + 2.0 ** -21 * (t.gather(1, order) + h[:, None] + 1)
        assert bool(((top.double() == want) | ((top.double() - want).abs() <= tol)).all()), "%s: top log probabilities" % what


def _run_logprobs(x, scale=1.0, targets=None, k=0, entropy=True):
    rows, V = x.shape
    ws = torch.full((nwc.nwc_token_logprobs_workspace_size(rows, V, k),), 255, dtype=torch.uint8, device="cuda")
    lp = None if targets is None else torch.full(targets.shape, 7.0, device="cuda")
    ent = torch.full((rows,), 7.0, device="cuda") if entropy else None
    ids = torch.full((rows, k), -9, dtype=torch.int32, device="cuda") if k else None
    top = torch.full((rows, k), 7.0, device="cuda") if k else None
    call = nwc.TokenLogprobs(x, ws, targets=targets, logprobs=lp, entropy=ent, top_ids=ids, top_logprobs=top, scale=scale)
    nwc.nwc_token_logprobs(call)
    torch.cuda.synchronize()
    first = [None if o is None else o.clone() for o in (lp, ent, ids, top)]
    nwc.nwc_token_logprobs(call)
    torch.cuda.synchronize()
    for a, b in zip(first, (lp, ent, ids, top)):
        assert a is None or torch.equal(a.view(torch.int32), b.view(torch.int32))
    return lp, ent, ids, top


LP_CASES = [  # rows, vocab, k, targets, scale
    (1, 1, 1, 1, 1.0), (1, 7, 7, 2, 1.0), (3, 64, 64, 1, 0.7), (2, 1001, 20, 3, 1.0), (1, 128256, 20, 1, 1.0),
    (1, 128256, 64, 1, 2.0), (5, 32003, 5, 4, 1.0), (16, 128256, 20, 1, 1.0), (64, 50000, 1, 1, 1.3), (600, 1001, 10, 2, 1.0),
    (520, 12289, 33, 1, 1.0), (9, 4097, 64, 1, 1.0), (1, 4103, 50, 1, 1.0), (2, 300007, 20, 1, 1.0), (700, 8, 8, 1, 1.0)]


@pytest.mark.parametrize("case", LP_CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("f32", [False, True])
def test_logprobs(case, f32):
    rows, V, k, n, scale = case
    _say("logprobs %s f32 %s" % (case, f32))
    g = torch.Generator(device="cuda").manual_seed(rows + V)
    ld = (V + 7) // 8 * 8 + (16 if rows > 1 else 0)
    x = (3 * torch.randn((rows, ld), generator=g, device="cuda")).to(torch.float32 if f32 else torch.bfloat16)
    x[:, V:] = float("nan")                                    # between the rows
    x = x[:, :V]
    targets = torch.randint(0, V, (rows, n), generator=g, device="cuda", dtype=torch.int32)
    if rows > 1:
        targets[0, 0], targets[-1, -1] = -1, V                 # no token
    _check_logprobs(x, scale, targets, *_run_logprobs(x, scale, targets, k), "plain")
    # parts of what can be asked for
    _check_logprobs(x, scale, targets, *_run_logprobs(x, scale, targets, 0, False), "targets alone")
    _check_logprobs(x, scale, None, *_run_logprobs(x, scale, None, k, False), "top alone")
    _check_logprobs(x, scale, None, *_run_logprobs(x, scale, None, 0, True), "entropy alone")


@pytest.mark.parametrize("rows", [1, 3, 600])
@pytest.mark.parametrize("f32", [False, True])
def test_logprobs_orders_ties_and_masks(rows, f32):
    V, k = 20000, 20
    dt = torch.float32 if f32 else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(5)
    lowest = torch.finfo(dt).min
    kinds = {
        "all equal": torch.zeros((rows, V), device="cuda"),
        "signed zeros": torch.where(torch.arange(V, device="cuda") % 2 == 0, -0.0, 0.0).repeat(rows, 1),
        "few values": torch.randint(0, 3, (rows, V), generator=g, device="cuda").float(),
        "rising": (torch.arange(V, device="cuda") / V * 50).repeat(rows, 1),
        "falling": (-torch.arange(V, device="cuda") / V * 50).repeat(rows, 1),
        "masked to three": torch.full((rows, V), -float("inf"), device="cuda"),
        "masked by the lowest": torch.full((rows, V), lowest, device="cuda"),
        "one token": torch.full((rows, V), -float("inf"), device="cuda"),
        "two far": torch.randn((rows, V), generator=g, device="cuda"),
        "nothing but the lowest": torch.full((rows, V), lowest, device="cuda")}
    kinds["masked to three"][:, [17, 4000, 19999]] = 1.0
    kinds["masked by the lowest"][:, [5, 6, 15000]] = torch.tensor([1.0, 2.0, 3.0], device="cuda")
    kinds["one token"][:, 12345] = -3.0
    kinds["two far"][:, [3, 19998]] += 300.0
    for name, x in kinds.items():
        _say("logprobs %s %d rows" % (name, rows))
        x = x.to(dt)
        targets = torch.randint(0, V, (rows, 2), generator=g, device="cuda", dtype=torch.int32)
        targets[:, 0] = 17
        for k in (1, 20, 64):
            _check_logprobs(x, 1.0, targets, *_run_logprobs(x, 1.0, targets, k), name)


@pytest.mark.parametrize("rows", [1, 600])
def test_logprobs_of_odd_rows(rows):
    V, k = 9000, 6
    x = torch.randn((rows, V), generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    targets = torch.full((rows, 1), 4, dtype=torch.int32, device="cuda")
    empty = torch.full((rows, V), -float("inf"), device="cuda")
    lp, ent, ids, top = _run_logprobs(empty, 1.0, targets, k)
    assert bool((lp == -float("inf")).all()) and bool((ent == 0).all()) and bool((top == -float("inf")).all())
    assert torch.equal(ids, torch.arange(k, device="cuda", dtype=torch.int32).repeat(rows, 1))
    for value in (float("nan"), float("inf")):
        y = x.clone()
        y[:, 7777] = value
        y[:, 8888] = value
        lp, ent, ids, top = _run_logprobs(y, 1.0, targets, k)
        assert bool(lp.isnan().all()) and bool(ent.isnan().all()) and bool(top.isnan().all())
        z = x.clone()
        z[:, 7777] = z[:, 8888] = 1e30
        assert torch.equal(ids.long(), torch.sort(z, dim=-1, descending=True, stable=True).indices[:, :k])
    # a row of NaN leaves the others as they are
    if rows > 1:
        y = x.clone()
        y[5] = float("nan")
        lp, ent, ids, top = _run_logprobs(y, 1.0, targets, k)
        others = [r for r in range(rows) if r != 5]
        _check_logprobs(y[others], 1.0, targets[others], lp[others], ent[others], ids[others], top[others], "beside a row of NaN")


def test_logprobs_captured_and_on_two_streams():
    V, k = 128256, 20
    g = torch.Generator(device="cuda").manual_seed(8)
    xs = [torch.randn((rows, V), generator=g, device="cuda").to(torch.bfloat16) for rows in (1, 4)]
    bufs = []
    for x in xs:
        rows = x.shape[0]
        ws = torch.empty(nwc.nwc_token_logprobs_workspace_size(rows, V, k), dtype=torch.uint8, device="cuda")
        o = (torch.empty(rows, device="cuda"), torch.empty((rows, k), dtype=torch.int32, device="cuda"), torch.empty((rows, k), device="cuda"))
        bufs.append((o, nwc.TokenLogprobs(x, ws, entropy=o[0], top_ids=o[1], top_logprobs=o[2])))
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        nwc.nwc_token_logprobs(bufs[0][1], stream=streams[0])
    for i in range(4):
        for x in xs:
            x.copy_(torch.randn(x.shape, generator=g, device="cuda").to(torch.bfloat16))
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[0]):
            graph.replay()
        nwc.nwc_token_logprobs(bufs[1][1], stream=streams[1])
        torch.cuda.synchronize()
        for x, (o, _) in zip(xs, bufs):
            _check_logprobs(x, 1.0, None, None, *o, "replay %d" % i)


def test_residual_captured():
    g = torch.Generator(device="cuda").manual_seed(9)
    x, y = (torch.randn((3, 2560), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.ones(2560, dtype=torch.bfloat16, device="cuda")
    out, x_out = torch.empty_like(x), torch.empty_like(x)
    call = nwc.ResidualNorm(x, y, x_out=x_out, out=out, weight=w, y_weight=w)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        nwc.nwc_residual_norm(call, stream=stream)
    for _ in range(3):
        y.copy_(torch.randn(y.shape, generator=g, device="cuda").to(torch.bfloat16))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        _check_residual(_ref_residual(x, y, w, None, 1.0, w), x_out, out, w, "replay", True)


def test_refusals_of_device_tensors():
    bf, f, i = torch.bfloat16, torch.float32, torch.int32
    z = lambda shape, dtype: torch.zeros(shape, dtype=dtype, device="cuda")
    x, y, w, out = z((4, 64), bf), z((4, 64), bf), z(64, bf), z((4, 64), bf)
    for kw in (dict(y=z((4, 64), f)), dict(y=z((3, 64), bf)), dict(y=y, gate=z((4, 32), bf)), dict(y=y, gate=w, y_weight=z(63, bf)),
               dict(out=out), dict(weight=w), dict(y=y, x_out=z((4, 64), f)), dict(out=out.T, weight=w), dict(gate=w, out=out, weight=w),
               dict(y=y, x_out=x.clone(), keep=False)):
        with pytest.raises((ValueError, TypeError)):
            nwc.ResidualNorm(x, **kw)
    for bad in (nwc.ResidualNorm(x, y, eps=-1.0), nwc.ResidualNorm(x, y, scale=float("inf")), nwc.ResidualNorm(x, out=w.view(1, 64).expand(4, 64), weight=w),
                nwc.ResidualNorm(z((4, 60), bf), z((4, 60), bf))):
        with pytest.raises(nwc.NwcError):
            nwc.nwc_residual_norm(bad)
    logits, ws = z((4, 1000), bf), z(nwc.nwc_token_logprobs_workspace_size(4, 1000, 5), torch.uint8)
    t, lp, ent, ids, top = z((4, 2), i), z((4, 2), f), z(4, f), z((4, 5), i), z((4, 5), f)
    for kw in (dict(targets=t), dict(logprobs=lp), dict(targets=t.long(), logprobs=lp), dict(targets=t, logprobs=lp[:, :1]),
               dict(entropy=ent[:3]), dict(top_ids=ids), dict(top_ids=ids, top_logprobs=top.to(bf)), dict(top_ids=ids[:, ::2], top_logprobs=top[:, ::2])):
        with pytest.raises((ValueError, TypeError)):
            nwc.TokenLogprobs(logits, ws, **kw)
    with pytest.raises((ValueError, TypeError)):
        nwc.TokenLogprobs(logits.half(), ws, entropy=ent)
    for bad in (nwc.TokenLogprobs(logits, ws), nwc.TokenLogprobs(logits, ws, entropy=ent, scale=0.0),
                nwc.TokenLogprobs(logits[:, 1:], ws, entropy=ent), nwc.TokenLogprobs(logits, ws[:128], entropy=ent),
                nwc.TokenLogprobs(z((4, 1001), bf), ws, entropy=ent),
                nwc.TokenLogprobs(logits, ws, top_ids=z((4, 65), i), top_logprobs=z((4, 65), f))):
        with pytest.raises(nwc.NwcError):
            nwc.nwc_token_logprobs(bad)
