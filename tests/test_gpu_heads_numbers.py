"""Norm and rotation of heads at the ends of their numbers' range.

Tolerances as for ordinary heads, from the roundings: the result's, 2^-8 |out|
(BF16: half a step), and 2^-16 of the pair's two components for about ten
roundings in FP32 and the hardware's sine and cosine, allowed 2^-17 each.
"""
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
