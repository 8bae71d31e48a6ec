"""Norm and rotation of heads at the ends of their numbers' range.

Tolerances as for ordinary heads, from the roundings: the result's, 2^-8 |out|
(BF16: half a step), and 2^-16 of the pair's two components for about ten
roundings in FP32 and the hardware's sine and cosine, allowed 2^-17 each.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import decode_gemv_byte_amd as nwc  # noqa: E402
from test_gpu_attention import _check_heads, _freqs, _i32, _ref_heads, _say  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
@pytest.mark.parametrize("d", [8, 64, 128, 200, 256])
def test_norm_of_heads_of_any_size(d, eps):
    # heads whose squares, or whose squares' sum, pass FP32's range at either end; the last token mixes sizes
    _say("norm of heads of any size %d %g" % (d, eps))
    g = torch.Generator(device="cuda").manual_seed(d)
    exponents = [-120, -100, -80, -64, -50, -30, 0, 30, 58, 62, 64, 80, 100, 120, 125]
    x = torch.randn((len(exponents) + 1, 3, d), generator=g, device="cuda").clamp(-3, 3)
    for t, e in enumerate(exponents):
        x[t] *= 2.0 ** e
    x[-1, :, ::3] *= 2.0 ** 100
    x = x.to(torch.bfloat16)
    w = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
    pos, freqs = _i32(range(len(x))), _freqs(d // 2 // 8 * 8)
    out = torch.empty_like(x)
    nwc.nwc_qk_norm_rope(nwc.QkNormRope(x, None, pos, q_out=out, q_weight=w, eps=eps, freqs=freqs))
    torch.cuda.synchronize()
    # eps as the call takes it, an FP32 number
    ref, size = _ref_heads(x, w, pos, freqs, "half", eps=float(torch.tensor(eps, dtype=torch.float32)))
    _check_heads(out, ref, size, "heads")


@pytest.mark.parametrize("style", ["half", "pairs"])
def test_angles_of_frequencies_above_one(style):
    # position * frequency to 2^31 * 1000 radians: the stated 3 2^-53 of it, in sine and cosine both, of the pair's components
    _say("angles of frequencies above one %s" % style)
    d = 64
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((300, 2, d), generator=g, device="cuda").to(torch.bfloat16)
    freqs = torch.rand(d // 2, generator=g, device="cuda") * torch.tensor([1.0, 30.0, 1000.0, 1e-3], device="cuda").repeat(d // 8)
    pos = torch.randint(0, 2 ** 31 - 1, (300,), generator=g, device="cuda").to(torch.int32)
    pos[:2] = _i32([2 ** 31 - 1, 0])
    out = torch.empty_like(x)
    nwc.nwc_qk_norm_rope(nwc.QkNormRope(x, None, pos, q_out=out, freqs=freqs, style=style))
    torch.cuda.synchronize()
    # the product exactly (55 bits) and its reduction with 64 bits of 2 pi, 2^-64 of the angle
    angle = np.outer(pos.cpu().numpy().astype(np.longdouble), freqs.cpu().numpy().astype(np.longdouble))
    two_pi = 2 * np.longdouble("3.14159265358979323846264338327950288")
    turn = torch.from_numpy(np.float64(angle - np.rint(angle / two_pi) * two_pi)).cuda()[:, None]
    i, j = (slice(0, d // 2), slice(d // 2, d)) if style == "half" else (slice(0, d, 2), slice(1, d, 2))
    a, b = x.double()[..., i], x.double()[..., j]
    off = 3 * 2.0 ** -53 * torch.from_numpy(np.float64(angle)).cuda()[:, None]
    for part, ref in ((i, a * turn.cos() - b * turn.sin()), (j, b * turn.cos() + a * turn.sin())):
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -16 + off) * (a.abs() + b.abs())
        assert bool(((out.double()[..., part] - ref).abs() <= tol).all())


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("d", [8, 64, 72, 128, 256])
def test_norm_of_heads_of_different_sizes_in_a_token(d, eps):
    # heads that one wavefront takes together, some of them past the range and some not; queries and keys, with and without norm
    _say("norm of different heads %d %g" % (d, eps))
    g = torch.Generator(device="cuda").manual_seed(d + 1)
    exponents = torch.tensor([0, 100, -120, 3, 64, -64, -5, 120, 1, -100, 80], device="cuda").double()
    x = torch.randn((70, 11, d), generator=g, device="cuda").clamp(-3, 3).double()
    turn = (torch.arange(70, device="cuda")[:, None] + torch.arange(11, device="cuda")) % 11
    x = (x * 2.0 ** exponents[turn][..., None]).to(torch.bfloat16)
    q, k = x[:, :7].contiguous(), x[:, 7:].contiguous()
    w = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
    pos, freqs = _i32(range(70)), _freqs(8)
    for weights in ((w, w), (w, None), (None, w)):
        q_out, k_out = torch.empty_like(q), torch.empty_like(k)
        nwc.nwc_qk_norm_rope(nwc.QkNormRope(q, k, pos, q_out=q_out, k_out=k_out, q_weight=weights[0], k_weight=weights[1], eps=eps,
                                            freqs=freqs))
        torch.cuda.synchronize()
        for name, src, out, weight in (("q", q, q_out, weights[0]), ("k", k, k_out, weights[1])):
            ref, size = _ref_heads(src, weight, pos, freqs, "half", eps=float(torch.tensor(eps, dtype=torch.float32)))
            # heads that are not normed reach below 2^-126, where BF16's numbers are 2^-133 apart: half of that beside the
            # relative bounds
            err = (out.double() - ref).abs()
            assert bool((err <= 2.0 ** -8 * ref.abs() + 2.0 ** -16 * size + 2.0 ** -134).all()), name
