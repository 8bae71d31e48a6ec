"""How attention over the paged cache splits its work: plans of many rows and
groups, ranges of many units, items cut between workgroups.  In long rows of
random values a lost unit drowns in the tolerance, so here every unit shows.

Tolerances as in test_gpu_attention_numbers.py: 2^-8 |out| for the output's
rounding, 2^-16 sum w |v| for the weights', 2^-10 sum w |v| for FP32.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from test_gpu_attention import _Batch, _say  # noqa: E402
from test_gpu_attention_numbers import _check, _run, _slots  # noqa: E402

pytestmark = pytest.mark.gpu

# rows, groups: (first row, end, shared length)
PLANS = {
    "257 rows": ([37 - r % 38 for r in range(257)], [(0, 100, 8), (100, 256, 17)]),
    "300 rows, no groups": ([r % 45 for r in range(300)], []),
    "600 rows, 3 groups": ([40 - r % 7 for r in range(600)], [(0, 250, 33), (250, 251, 20), (251, 599, 30)]),
    "64 rows, 63 groups": ([20 + r for r in range(64)], [(r, r + 1, 18) for r in range(62)] + [(62, 64, 40)]),
    "64 rows, 64 groups": ([20 + r for r in range(64)], [(r, r + 1, 18) for r in range(64)]),
    "60 rows, 100 groups": ([50 - r % 30 for r in range(60)], [(r // 5 * 3, (r // 5 + 1) * 3 if r % 5 == 4 else r // 5 * 3, 19) for r in range(100)]),
    "65 rows, 512 groups": ([30 + r % 3 for r in range(65)], [(r // 8, (r + 1) // 8, 25) for r in range(512)]),
    "4096 rows, 128 groups": ([(r * 2654435761 >> 7) % 41 - 1 for r in range(4096)], [(i * 32, i * 32 + 32, 8) for i in range(128)]),
    "4096 rows, 512 groups": ([(r * 2654435761 >> 9) % 30 + 1 for r in range(4096)], [(i * 8, i * 8 + 8, 11) for i in range(512)]),
}


@pytest.mark.parametrize("hq,hk,d,page", [(4, 2, 64, 16), (8, 1, 128, 16)])
@pytest.mark.parametrize("name", list(PLANS))
def test_plans_of_many_rows_and_groups(name, hq, hk, d, page):
    # a table that covers too much for the launch of short tables
    lengths, groups = PLANS[name]
    _say("plan %s, %d %d %d" % (name, hq, hk, d))
    b = _Batch(lengths, hq, hk, d, page, groups, seed=len(lengths), covers=4000)
    _run(b)
    _check(b, name)
    first = b.out.clone()
    b.out.fill_(7.0)
    _run(b)
    assert torch.equal(b.out, first), "not the same bits"


def _every_unit(b, what):
    """Equal weights, and of a unit of 32 positions the ones in one component (another one for each key-value head): a unit left
    out or taken twice changes its component by a share that no rounding has."""
    _, hk, _, d = b.vp.shape
    b.q.zero_()
    for r, n in enumerate(b.lengths):
        if n > 0:
            pages, slots = _slots(b, r)
            of = (torch.arange(int(n), device="cuda")[:, None] // 32 + 7 * torch.arange(hk, device="cuda")) % d
            b.vp[pages, :, slots] = torch.nn.functional.one_hot(of, d).to(torch.bfloat16)
    _run(b)
    _check(b, what + ", every unit")


def _single_positions(b, what, seed):
    """A few positions take nearly all of the weight: first, last, on unit borders, anywhere."""
    _, hk, _, d = b.vp.shape
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = np.random.default_rng(seed)
    b.q.fill_(1.0)
    for x in (b.kp, b.vp):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda", dtype=torch.bfloat16) * (0.01 if x is b.kp else 1))
    shared = int(b.groups[1][0]) if b.groups[0] is not None else 0
    planted = {}
    for r, n in enumerate(b.lengths):
        if n > 0:
            pages, slots = _slots(b, r)
            at = rnd.integers(0, n, 6).tolist() + [n - 1] + [int(x) // 32 * 32 - 1 for x in rnd.integers(32, max(n, 33), 3) if x < n]
            # positions of the prefix are the same for all of its rows, in copied pages too
            at = [x for x in at if x >= shared] + planted.setdefault("shared", [x for x in at if x < shared])
            at = torch.tensor(sorted(set(at)), device="cuda")
            score = 12.0 + (at % 5).float() * 0.3
            b.kp[pages[at], :, slots[at]] = (score / d / b.scale).to(torch.bfloat16)[:, None, None].expand(len(at), hk, d)
            if shared and r:
                first = [x[:shared] for x in _slots(b, 0)]
                for x in (b.kp, b.vp):
                    x[pages[:shared], :, slots[:shared]] = x[first[0], :, first[1]]
    _run(b)
    _check(b, what + ", single positions")


@pytest.mark.parametrize("rows", [2, 5, 12])                     # 16, 40 and 96 columns
@pytest.mark.parametrize("d,page", [(64, 32), (96, 16), (128, 64), (192, 128), (256, 32)])
def test_prefix_of_many_units(d, page, rows):
    # 751 units in each of 8 key-value heads, 24 for each of 256 workgroups: rings go round, and pages end inside units
    _say("prefix of many units %d %d" % (d, rows))
    shared = 24005
    lengths = [shared + 1 + 37 * r for r in range(rows)]
    b = _Batch(lengths, 8 * 8, 8, d, page, [(0, rows, shared)], seed=d + rows)
    _every_unit(b, "prefix")
    _single_positions(b, "prefix", d + rows)


LONG = {"one row": [40001], "a longer one": [100003], "ragged": [9000 - 211 * r for r in range(40)], "few": [9001, 1, 8192, 77]}


@pytest.mark.parametrize("name", list(LONG))
@pytest.mark.parametrize("hq,hk,d,page", [(16, 4, 64, 32), (20, 4, 96, 16), (32, 8, 128, 64), (10, 5, 192, 128), (8, 2, 256, 32),
                                          (40, 2, 128, 16), (80, 2, 64, 16), (64, 1, 256, 64)])
def test_own_positions_of_many_units(hq, hk, d, page, name):
    _say("own positions of many units %s %d %d %d" % (name, hq, hk, d))
    b = _Batch(LONG[name], hq, hk, d, page, seed=d + hq)
    _every_unit(b, name)
    _single_positions(b, name, d + hq)


@pytest.mark.parametrize("hq,hk,d,page", [(16, 4, 64, 32), (20, 4, 96, 16), (32, 8, 128, 64), (10, 5, 192, 128), (8, 2, 256, 32),
                                          (40, 2, 128, 16)])
def test_short_tables_of_many_units(hq, hk, d, page):
    # the launch of short tables: as many rows as it takes for the widest table, several units a wavefront
    _say("short tables of many units %d %d %d" % (hq, hk, d))
    rows = 128 // hk + 1
    b = _Batch([1024 - 15 * r % 700 for r in range(rows)], hq, hk, d, page, seed=d + hq)
    _every_unit(b, "short tables")
    _single_positions(b, "short tables", d + hq)


def test_the_checks_see_a_lost_unit():
    # the reference without one page of 16 positions, or without the last 32: each check says so
    b = _Batch([40001], 8, 2, 128, 16, seed=1)
    for fill, gone in ((_every_unit, 1234), (_every_unit, None), (lambda b, what: _single_positions(b, what, 3), None)):
        fill(b, "as it is")
        table, lengths = b.table.copy(), b.lengths.copy()
        if gone is None:
            b.lengths = b.lengths - 32
        else:
            b.table[0, gone] = -1
        with pytest.raises(AssertionError):
            _check(b, "with a part left out of the reference")
        b.table, b.lengths = table, lengths
