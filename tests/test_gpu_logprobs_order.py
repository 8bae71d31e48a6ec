"""The k most likely tokens of rows that hold NaN, infinities or both, at any place,
the first token and whole rows among them; rows by one workgroup and by several."""
import pytest
import torch

import decode_gemv_byte_amd as nwc

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def _top(x, k):
    rows, V = x.shape
    ws = torch.empty(nwc.nwc_token_logprobs_workspace_size(rows, V, k), dtype=torch.uint8, device="cuda")
    ent, top = torch.empty(rows, device="cuda"), torch.empty((rows, k), device="cuda")
    ids = torch.full((rows, k), -7, dtype=torch.int32, device="cuda")
    nwc.nwc_token_logprobs(nwc.TokenLogprobs(x, ws, entropy=ent, top_ids=ids, top_logprobs=top))
    torch.cuda.synchronize()
    return ids.long(), top, ent


def _order(x, k):
    """NaN above +infinity above all finite values; of equal ones the lower index first."""
    z = x.double()
    z = torch.where(z == INF, torch.full_like(z, 1e300), z)
    return torch.sort(torch.where(z.isnan(), torch.full_like(z, 1e301), z), dim=-1, descending=True, stable=True).indices[:, :k]


PLACES = [[0], [0, 1], [0, 2], [1], [0, -1], [-1], [0, 1, 2, 3, 4], [7, 8]]


@pytest.mark.parametrize("places", PLACES, ids=str)
@pytest.mark.parametrize("rows,V,k", [(1, 5, 3), (2, 9, 9), (3, 64, 64), (1, 4097, 20), (1, 20000, 64), (600, 9000, 6), (2, 128256, 20)])
@pytest.mark.parametrize("f32", [False, True])
def test_nan_stands_first(rows, V, k, places, f32):
    print("nan at %s of %d x %d, k %d, f32 %s" % (places, rows, V, k, f32), flush=True)
    g = torch.Generator(device="cuda").manual_seed(V)
    dt = torch.float32 if f32 else torch.bfloat16
    x = torch.full((rows, (V + 7) // 8 * 8), NAN, dtype=dt, device="cuda")[:, :V]
    for others in (3 * torch.randn((rows, V), generator=g, device="cuda"), torch.zeros((rows, V), device="cuda"),
                   torch.full((rows, V), -INF, device="cuda"), torch.full((rows, V), INF, device="cuda")):
        x.copy_(others.to(dt))
        at = [p % V for p in places]
        x[:, at] = NAN
        ids, top, ent = _top(x, k)
        assert torch.equal(ids, _order(x, k))
        assert bool(top.isnan().all()) and bool(ent.isnan().all())


@pytest.mark.parametrize("rows,V,k", [(1, 1, 1), (1, 5, 5), (3, 7, 7), (4, 64, 64), (1, 4097, 64), (2, 20000, 20), (600, 1001, 10), (1, 128256, 20)])
@pytest.mark.parametrize("f32", [False, True])
def test_rows_of_nan_throughout(rows, V, k, f32):
    print("%d rows of %d NaN, k %d, f32 %s" % (rows, V, k, f32), flush=True)
    bits = torch.tensor([0x7FC00000, 0x7F800001, -1, -0x400000], dtype=torch.int64).to(torch.int32)   # NaN of any sign and payload
    x = bits.view(torch.float32).repeat(rows * ((V + 7) // 8 * 2)).view(rows, -1).cuda()[:, :V]
    if not f32:
        x = torch.tensor([0x7FC0, 0x7F81, -1, -0x40], dtype=torch.int16).view(torch.bfloat16).repeat(rows * ((V + 7) // 8 * 2)).view(rows, -1).cuda()[:, :V]
    ids, top, ent = _top(x, k)
    assert torch.equal(ids, torch.arange(k, device="cuda").repeat(rows, 1))
    assert bool(top.isnan().all()) and bool(ent.isnan().all())


@pytest.mark.parametrize("f32", [False, True])
def test_infinities_and_one_part_with_nan(f32):
    V, k = 20000, 20        # five parts
    dt = torch.float32 if f32 else torch.bfloat16
    for part in range(5):
        x = torch.randn((2, V), generator=torch.Generator(device="cuda").manual_seed(part), device="cuda").to(dt)
        first = part * V // 5 // 8 * 8
        x[0, first] = NAN
        x[0, [3, 9000]] = INF
        x[1, first:first + 30] = INF
        ids, top, ent = _top(x, k)
        assert torch.equal(ids, _order(x, k)), part
