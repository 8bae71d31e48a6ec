"""Chunk attention whose outputs count positions: every position's weight is the same
(queries of zero), and a value is one in a single component that tells where the
position lies.  Component e of a token that sees n positions is then c_e / n, c_e
the number of its positions that name e: a unit lost, counted twice or seen too early
changes a component by more than its tolerance, at any length.

Weights are all 1, a power of two: their rounding to BF16 and the sums of ones are
exact.  What is left: the quotient, the parts' means and the sums over at most 256
parts in FP32 (2^-24 each, of sums of numbers that are none below zero: 2^-15 in all),
and the output's rounding: (2^-8 + 2^-15) of the value."""
import numpy as np
import pytest
import torch

from test_gpu_chunk import Case, _say
import decode_gemv_byte_amd as nwc

pytestmark = pytest.mark.gpu


def _counting(c, key):
    """Values that are one in component key(position) of their head dimension; keys of any kind, queries of zero."""
    c.q_all.zero_()
    c.v.zero_()
    for r in range(len(c.new)):
        at = np.arange(max(0, int(c.lengths[r])))
        pg = torch.from_numpy(c.table[r, at // c.page]).cuda()
        c.v[pg, :, torch.from_numpy(at % c.page).cuda(), torch.from_numpy(key(at) % c.d).cuda()] = 1.0


def _check(c, key, what):
    left = torch.ones(c.out.shape[0], dtype=torch.bool, device="cuda")
    for r in range(len(c.new)):
        n, length, t0 = int(c.new[r]), int(c.lengths[r]), int(c.start[r])
        hits = torch.zeros((length, c.d), dtype=torch.float64, device="cuda")
        at = np.arange(length)
        hits[torch.from_numpy(at).cuda(), torch.from_numpy(key(at) % c.d).cuda()] = 1.0
        seen = torch.arange(length - n + 1, length + 1, device="cuda")
        want = (hits.cumsum(0)[length - n:] / seen[:, None])[:, None].expand(n, c.hq, c.d)
        err = (c.out[t0:t0 + n].double() - want).abs()
        bad = ~(err <= (2.0 ** -8 + 2.0 ** -15) * want)
        assert not bool(bad.any()), "%s, row %d: %d outside, first %s" % (what, r, int(bad.sum()), bad.nonzero()[0].tolist())
        left[t0:t0 + n] = False
    assert bool((c.out[left] == 7.0).all())


# a unit's positions in one component (64 or 32 of them), or all positions in turn, or half a unit
KEYS = {"units of 64": lambda p: p // 64, "units of 32": lambda p: p // 32, "positions": lambda p: p, "pages of 16": lambda p: p // 16}
CASES = [  # new, lengths, q heads, kv heads, head_dim, page
    ([70], [40000], 8, 2, 128, 64), ([64], [131071], 32, 8, 128, 64), ([1500, 3], [9000, 20001], 32, 8, 128, 128),
    ([5], [512], 32, 8, 128, 64), ([4100], [4100], 8, 2, 128, 64), ([8] * 4, [3000, 3001, 4095, 7777], 32, 8, 128, 32),
    ([1] * 31 + [512], [131 * i + 1 for i in range(31)] + [4001], 32, 8, 128, 32),
    ([1] * 31 + [512], [131 * i + 1 for i in range(31)] + [4001], 64, 8, 64, 32), ([300], [30011], 64, 8, 64, 16),
    ([77, 500], [30011, 2000], 20, 4, 96, 64), ([333, 40], [1000, 25003], 10, 5, 192, 64), ([129, 65], [12345, 30011], 8, 2, 256, 32)]


@pytest.mark.parametrize("key", list(KEYS), ids=lambda k: k.replace(" ", "-"))
@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s-%s-%d-%d-%d-%d" % ((sum(c[0]), max(c[1])) + c[2:]))
def test_every_position_counts_once(case, key):
    _say("counting %s by %s" % (case, key))
    c = Case(*case, seed=11)
    _counting(c, KEYS[key])
    nwc.nwc_attend_chunk(c.call())
    torch.cuda.synchronize()
    _check(c, KEYS[key], key)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s-%s-%d-%d-%d-%d" % ((sum(c[0]), max(c[1])) + c[2:]))
def test_a_token_sees_up_to_its_own_position(case):
    """Values are ones at each new token's own position, in its own component, and twos behind the row's last."""
    _say("own positions %s" % (case,))
    c = Case(*case, seed=12)
    c.q_all.zero_()
    c.v.fill_(2.0)
    for r in range(len(c.new)):
        n, length = int(c.new[r]), int(c.lengths[r])
        at = np.arange(length)
        pg, slot = torch.from_numpy(c.table[r, at // c.page]).cuda(), torch.from_numpy(at % c.page).cuda()
        c.v[pg, :, slot] = 0.0
        own = at >= length - n
        c.v[pg[torch.from_numpy(own)], :, slot[torch.from_numpy(own)], torch.from_numpy(at[own] % c.d).cuda()] = 1.0
    nwc.nwc_attend_chunk(c.call())
    torch.cuda.synchronize()
    for r in range(len(c.new)):
        n, length, t0 = int(c.new[r]), int(c.lengths[r]), int(c.start[r])
        pos = torch.arange(length - n, length, device="cuda")
        hits = torch.zeros((n, c.d), dtype=torch.float64, device="cuda")
        hits[torch.arange(n, device="cuda"), pos % c.d] = 1.0
        want = (hits.cumsum(0) / (pos + 1)[:, None])[:, None].expand(n, c.hq, c.d)
        err = (c.out[t0:t0 + n].double() - want).abs()
        assert bool((err <= (2.0 ** -8 + 2.0 ** -15) * want).all()), r
