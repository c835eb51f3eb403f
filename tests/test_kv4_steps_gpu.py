"""Attention over a cache whose scores rise in steps along a sequence: once, in a single row, again
and again, up and back, or slowly and then at once; by a few tens of nats to hundreds, at every
place of an item, over value rows of scales that stay, fall and rise.  Batches that give a CTA
whole items of many units, so that the running references move within a CTA, and its queues
come round.

Tolerance as in test_kv4_gpu.py, u |o| + (u + 2^-10) A + 2^-23 W sum_j |v_j| / 2^e_j, and for the
scores' size, which passes the 2^6 that the 2^-10 allows for: a score, in log2 units, is a sum of
exact products in fp32, then goes through three roundings, so it is off by less than 8 * 2^-24 of
S = scale log2(e) sum |q| |k|; a weight by ln 2 times that, in the sum over the values and in the sum
of the weights: 2 ln 2 * 2^-21 S < 2^-20.5 S of A.
"""
import math

import pytest
import torch

from test_kv4_gpu import rows, table_of, two_to, values
from test_seq_gpu import DEV, U, gen, ints, normal, starts

pytestmark = pytest.mark.gpu

UNIT, EXTRA = 256, 2        # of the tcgen05 kernel: rows of a unit, units that an item costs besides
SCALE = 2.0 ** -6           # 16 elements of 4 a are a nats


def shares(lens, H):
    """How many units of an item each CTA of the tcgen05 kernel gets, by the documented split."""
    ways = torch.cuda.get_device_properties(0).multi_processor_count
    items = [-(-n // UNIT) for n in lens if n for _ in range(H)]
    total = sum(u + EXTRA for u in items)
    q, rem = divmod(total, ways)
    cuts = [q * w + min(w, rem) for w in range(1, ways + 1)]
    got, at, w = [], 0, 0
    for u in items:
        first, end = at + EXTRA, at + EXTRA + u
        while True:
            got.append(max(0, min(end, cuts[w]) - max(first, at)))
            if cuts[w] >= end:
                break
            at, w = cuts[w], w + 1
        at = end
        if cuts[w] == end:
            w += 1
    return got


def steps(kind, n, at, jump):
    """Nats by which the rows' scores lie above the rest."""
    i = torch.arange(n, device=DEV)
    up = (i >= at).float() * jump
    if kind == "row":
        return (i == at).float() * jump
    if kind == "again":
        return up + (i >= at + 300) * jump + (i >= at + 700) * jump
    if kind == "back":
        return up - (i >= at + 40) * jump
    if kind == "lag":
        return torch.where(i < at, (i / at) * 32.0, 32.0 + jump)
    return up


KINDS = ("once", "row", "again", "back", "lag")


def what_it_holds(cache, table, n, page):
    """Rows [n, H, D] in 64 bits, and 2^e of the value rows as ones of e4m3 elements."""
    i = torch.arange(n, device=DEV)
    where, slot = table.long()[i // page], i % page
    if cache.k_off is not None:
        k, v = (values(*(t[where, :, slot] for t in ts))
                for ts in ((cache.k, cache.k_exp, cache.k_off), (cache.v, cache.v_exp, cache.v_off)))
    else:
        k, v = (t[where, :, slot].double() * two_to(e.view(torch.uint8)[where, :, slot].long() - 127)[..., None]
                for t, e in ((cache.k, cache.k_exp), (cache.v, cache.v_exp)))
    lift = 6 if cache.k_off is not None else 0
    return k, v, two_to(cache.v_exp.view(torch.uint8)[where, :, slot].long() - 127 - lift)


def check(lib, lens, H, G, D, page, jump, dtype, width=None, seed=0):
    n_seq, T = len(lens), sum(lens)
    k, v = rows(seed, T, H, D), rows(seed + 1, T, H, D)
    first = 0
    for s, n in enumerate(lens):
        at = min(n - 1, UNIT * (1 + s % (n // UNIT)) + s * 53 % UNIT)
        part = slice(first, first + n)
        k[part, :, :16] = (steps(KINDS[s % len(KINDS)], n, at, jump) * 4)[:, None, None].to(k.dtype)
        unit = torch.arange(n, device=DEV) // UNIT
        tilt = (0.0, -5.0, 3.0)[s // len(KINDS) % 3]
        v[part] *= torch.exp2(tilt * unit)[:, None, None].to(v.dtype)
        first += n
    table, n_pages = table_of([-(-n // page) for n in lens], seed, width)
    cache = lib.make_kv_cache(n_pages, page, H, D, dtype=dtype)
    lib.kv_cache_append(cache, k, v, ints(lens), table, starts(lens))
    q = normal(gen(seed + 2), n_seq, H * G, D)
    # (heads that see the steps whole, by half, downwards, and not)
    q[:, :, :16] = torch.tensor([1.0, 0.5, -1.0, 0.0], device=DEV)[torch.arange(H * G, device=DEV) % 4,
                                                                   None].to(q.dtype)
    got = lib.paged_attention(q, cache, ints(lens), table, scale=SCALE)
    again = lib.paged_attention(q, cache, ints(lens), table, scale=SCALE)
    lib.sync_status()
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))
    for s, n in enumerate(lens):
        kk, vv, unit = what_it_holds(cache, table[s], n, page)
        qq = q[s].double().view(H, G, D)
        p = torch.softmax(torch.einsum("nhd,hgd->nhg", kk, qq) * SCALE, 0)
        size = torch.einsum("nhd,hgd->nhg", kk.abs(), qq.abs()).amax(0) * SCALE * math.log2(math.e)
        o, a = (torch.einsum("nhg,nhd->hgd", p, x) for x in (vv, vv.abs()))
        most = (p * unit[..., None]).amax(0)
        small = most[..., None] * (vv.abs() / unit[..., None]).sum(0)[:, None]
        bar = U * o.abs() + (U + 2.0 ** -10 + 2.0 ** -20.5 * size[..., None]) * a + 2.0 ** -23 * small
        mine = got[s].double().view(H, G, D)
        what = f"sequence {s} ({KINDS[s % len(KINDS)]})"
        assert torch.isfinite(mine).all(), f"{what}: not finite"
        over = (mine - o).abs() - bar
        assert (over <= 0).all(), f"{what}: over by {over.max().item():.3e}"


@pytest.mark.parametrize("dtype", [torch.uint8, torch.float8_e4m3fn])
@pytest.mark.parametrize("jump", [48, 64, 96, 256])
@pytest.mark.parametrize("G", [1, 4, 8, 16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("width", [None, 200])
def test_scores_in_steps(cuda_lib, D, G, jump, width, dtype):
    """A CTA gets items of eight units, whole as a rule: three more of each group's."""
    lens = [2000] * 64
    assert sorted(shares(lens, 8))[len(shares(lens, 8)) // 2] >= 6
    check(cuda_lib, lens, 8, G, D, 16, jump, dtype, width, seed=G + jump)


@pytest.mark.parametrize("dtype", [torch.uint8, torch.float8_e4m3fn])
@pytest.mark.parametrize("jump", [48, 96, 256])
@pytest.mark.parametrize("G", [2, 4, 5, 8])
@pytest.mark.parametrize("D", [64, 128])
def test_items_of_many_units(cuda_lib, D, G, jump, dtype):
    """A CTA gets 20 units of an item and more: the queues come round."""
    H = 8
    n_seq = torch.cuda.get_device_properties(0).multi_processor_count // H
    lens = [5632 - 37 * (s % 5) for s in range(n_seq)]
    assert max(shares(lens, H)) >= 20
    check(cuda_lib, lens, H, G, D, 64, jump, dtype, seed=G + jump + 1)
