"""The 8-bit key-value cache over the whole range of its scales: rows near the largest
finite value, rows whose scales lie further apart than fp32's exponents reach, rows of
zeros.  References, bounds and inputs as in test_seq_gpu.py; every case runs behind a
page table as long as the sequences and behind one that reaches further, which are
different kernels for 128-element heads."""
import math

import pytest
import torch

import test_seq_gpu as seq
from test_seq_gpu import DEV, close, fill, gen, ints, normal, rows_of, widened

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
BF16_MAX = torch.finfo(torch.bfloat16).max


def attended(lib, cache, narrow, lens, q, group, scale, what=""):
    """paged_attention behind both tables against the cache's rows in 64 bits; what lies
    beyond bf16's finite values saturates."""
    hkv = cache.heads
    for table in (narrow, widened(narrow, cache.page_size, hkv)):
        got = lib.paged_attention(q, cache, ints(lens), table, scale=scale)
        lib.sync_status()
        for s, n in enumerate(lens):
            k, v = rows_of(cache, narrow, s, n)
            see = torch.ones((1, n), dtype=torch.bool, device=DEV)
            for h in range(hkv * group):
                o, a = seq.attend_clean(q[s:s + 1, h], k[:, h // group], v[:, h // group], see,
                                        scale)
                close(got[s:s + 1, h], o.clamp(-BF16_MAX, BF16_MAX), a,
                      f"{what} sequence {s} of {n}, head {h}")
    return got


HEADS = [(64, 4), (64, 12), (128, 4), (128, 8), (128, 12)]


@pytest.mark.parametrize("D,group", HEADS)
def test_paged_values_near_the_largest(cuda_lib, D, group):
    """Value rows of up to 1.9 * 2^127: scales of 2^120, so that a weight that carries its
    row's scale and the sum of the weights without scales are 2^120 apart."""
    lens, scale = [3000, 300, 1], 1.5 * D ** -0.5

    def edit(k, v):
        v[:] = normal(gen(11), *v.shape) * 2.0 ** 125
        v[:, :, 0] = 1.9 * 2.0 ** 127
        v[::2, :, 0] *= -1
    cache, table, _, _ = fill(cuda_lib, lens, 64, 1, D, E4M3, seed=D + group, edit=edit)
    assert torch.all(cache.v_exp.view(torch.uint8)[table[0, 0]] == 247)
    attended(cuda_lib, cache, table, lens, normal(gen(1), 3, group, D), group, scale)


@pytest.mark.parametrize("D,group", HEADS)
@pytest.mark.parametrize("order", ["mixed", "rising", "falling"])
def test_paged_value_scales_beyond_fp32(cuda_lib, D, group, order):
    """Half of the value rows are 2^160 times the others: the small ones add nothing to the
    output, but their weights count in its denominator."""
    lens, scale = [2000, 130], D ** -0.5

    def edit(k, v):
        at = 0
        for n in lens:
            i = torch.arange(n, device=DEV)
            big = {"mixed": i % 2 == 0, "rising": i >= n // 2, "falling": i < n // 2}[order]
            v[at:at + n] *= torch.where(big, 2.0 ** 100, 2.0 ** -60)[:, None, None]
            at += n
    cache, table, _, _ = fill(cuda_lib, lens, 32, 1, D, E4M3, seed=D + group, edit=edit)
    attended(cuda_lib, cache, table, lens, normal(gen(2), 2, group, D), group, scale, order)


@pytest.mark.parametrize("D,group", HEADS)
@pytest.mark.parametrize("size", [1e-4, 1e-6, 1e-20])
def test_paged_value_rows_of_zeros(cuda_lib, D, group, size):
    """Rows of zeros (scale 1 by the cache's definition) among rows of small values: they
    add nothing to the output, and take no bits from the weights of the rows that do."""
    lens, scale = [1500, 70, 256], D ** -0.5

    def edit(k, v):
        v *= size
        v[::7] = 0
        v[1500 + 3:1500 + 60] = 0
        v[-1] = 0
    cache, table, _, _ = fill(cuda_lib, lens, 16, 1, D, E4M3, seed=group, edit=edit)
    attended(cuda_lib, cache, table, lens, normal(gen(3), 3, group, D), group, scale, size)


@pytest.mark.parametrize("D,group", HEADS)
def test_paged_value_row_of_zeros_takes_the_weight(cuda_lib, D, group):
    """The row with by far the largest score has a value of zeros (a sink): the output is
    small, and as exact as without it.  Rows of zeros and nothing else give zeros."""
    n, scale = 1100, D ** -0.5
    q = normal(gen(4), 2, group, D)
    q[:, :, 0] = 4.0

    def edit(k, v):
        k[:, :, 0] = 0
        for at in (0, 300, 301, 1099):  # scores of about 16 and 20 above the rest
            k[at] = 0
            k[at, :, 0] = 4 * scale ** -1 if at else 5 * scale ** -1
            v[at] = 0
        v[n:] = 0
    cache, table, _, _ = fill(cuda_lib, [n, 300], 32, 1, D, E4M3, seed=group, edit=edit)
    got = attended(cuda_lib, cache, table, [n, 300], q, group, scale)
    assert torch.all(got[1] == 0)


@pytest.mark.parametrize("D", [64, 128])
def test_cache_largest_values_come_back_finite(cuda_lib, D):
    """Magnitudes above 1.9375 * 2^127 round to 256 * 2^120 = 2^128, half a step beyond bf16's
    largest value: read back and attended to, they are that value, not an infinity."""
    n = 40
    x = torch.full((n, 1, D), BF16_MAX, dtype=torch.bfloat16, device=DEV)
    x[:, :, 1::2] = -BF16_MAX
    x[1, 0, 2], x[2, 0, 3] = 0.0, 1.875 * 2.0 ** 127
    x[3, 0, 4] = math.nan
    k = torch.zeros_like(x)
    cache = cuda_lib.make_kv_cache(3, 16, 1, D)
    table = ints([[2, 0, 1]])
    cuda_lib.kv_cache_append(cache, k, x, ints([n]), table, ints([0, n]))
    _, v = cuda_lib.kv_cache_gather(cache, table, ints([0, n]), total=n)
    cuda_lib.sync_status()
    want = rows_of(cache, table, 0, n)[1].clamp(-BF16_MAX, BF16_MAX)
    assert torch.isfinite(want).sum() == want.numel() - 1
    assert torch.equal(torch.isnan(v.double()), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(v.double()), torch.nan_to_num(want))
    # rows 0 and 1 alone: no NaN among them
    for group in (4, 8, 12):
        attended(cuda_lib, cache, table, [2], normal(gen(5), 1, group, D), group, D ** -0.5)
        attended(cuda_lib, cache, table, [1], normal(gen(5), 1, group, D), group, D ** -0.5)
