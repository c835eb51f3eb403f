"""Cases of the sequence operators that lie between the ones of test_seq_gpu.py: score and
value scales over 8-bit caches of 128-element heads (the tcgen05 kernel behind the wider
table), the bits of the weights, rows that are not finite, offsets beyond 32 bits, the
norm of many rows.  References and bounds as there, where nothing else is said."""
import math

import pytest
import torch

from test_seq_gpu import (DEV, DTYPES, U, attend, attend_clean, causal_mask, close, fill, gen,
                          ints, norm_reference, normal, paged_check, rows_of, starts, table_for,
                          widened)

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ one token over the cache
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("group", [4, 8])
@pytest.mark.parametrize("scale", [1e-4, 1.0, 3.0])
def test_paged_scales_of_wide_heads(cuda_lib, dtype, group, scale):
    paged_check(cuda_lib, [3000, 90, 257], 64, 1, group, 128, dtype, seed=4, scale=scale)


@pytest.mark.parametrize("group", [4, 8, 12])
@pytest.mark.parametrize("order", ["rising", "falling"])
def test_paged_value_scales_of_wide_heads(cuda_lib, group, order):
    """Value rows from 2^-60 to 2^60 over many units: m moves, and O with it, at each."""
    def edit(k, v):
        up = torch.exp2(torch.linspace(-60, 60, v.shape[0], device=DEV))
        v *= (up if order == "rising" else up.flip(0))[:, None, None]
    paged_check(cuda_lib, [2500], 32, 1, group, 128, E4M3, seed=5, edit=edit)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,group", [(64, 4), (128, 4), (128, 8)])
def test_paged_rising_scores(cuda_lib, dtype, D, group):
    """Every unit's scores far above the last one's."""
    def edit(k, v):
        k[:] = torch.arange(k.shape[0], device=DEV)[:, None, None] / 16.0
        k[:, :, 1::2] = 0
    cache, table, _, _ = fill(cuda_lib, [1500], 16, 1, D, dtype, seed=7, edit=edit)
    q = torch.ones((1, group, D), dtype=torch.bfloat16, device=DEV)
    q[:, 1::2] = 0.25
    see = torch.ones((1, 1500), dtype=torch.bool, device=DEV)
    k, v = rows_of(cache, table, 0, 1500)
    for t in (table, widened(table, 16, 1)):
        got = cuda_lib.paged_attention(q, cache, ints([1500]), t)
        cuda_lib.sync_status()
        for h in range(group):
            o, a = attend_clean(q[:, h], k[:, 0], v[:, 0], see, D ** -0.5)
            close(got[:, h], o, a, f"head {h}")


@pytest.mark.parametrize("D,bits,wide", [(128, 12, True), (128, 11, False), (64, 11, False)])
def test_paged_bits_of_the_weights(cuda_lib, D, bits, wide):
    """Two rows whose values cancel under the first head's weights, to what e4m3 leaves: the
    output's own rounding is small beside the weights'.  A weight is off by at most 2^-11
    (fp16) or 2^-12 (three e4m3 terms) of itself; scores and fp32 sums are off by less
    than 2^-14 (two terms of a query 2^-22 of its largest element, over 128 products; the
    exponential 2^-22)."""
    n, hkv, group = 64, 4, 4
    g = gen(30)
    table, n_pages = table_for([2] * n, 16)
    if wide:
        table = widened(table, 16, hkv)
    cache = cuda_lib.make_kv_cache(n_pages, 16, hkv, D)
    q, k = normal(g, n, hkv * group, D), normal(g, n, 2, hkv, D) * 0.5
    s = torch.einsum("nhd,nrhd->nrh", q[:, ::group].double(), k.double()) * D ** -0.5
    p = torch.softmax(s, 1)
    v = normal(g, n, 2, hkv, D)
    v[:, 1] = (-v[:, 0].double() * (p[:, 0] / p[:, 1])[..., None]).to(torch.bfloat16)
    cuda_lib.kv_cache_append(cache, k.view(2 * n, hkv, D), v.view(2 * n, hkv, D), ints([2] * n),
                             table, starts([2] * n))
    got = cuda_lib.paged_attention(q, cache, ints([2] * n), table).double()
    cuda_lib.sync_status()
    small = 0
    for b in range(n):
        kk, vv = rows_of(cache, table, b, 2)
        see = torch.ones((1, 2), dtype=torch.bool, device=DEV)
        for h in range(hkv * group):
            o, a = attend_clean(q[b:b + 1, h], kk[:, h // group], vv[:, h // group], see, D ** -0.5)
            bar = U * o.abs() + (2.0 ** -bits + 2.0 ** -14) * a
            assert ((got[b:b + 1, h] - o).abs() <= bar).all(), (b, h)
            small += int((o.abs() < a / 16).sum())
    assert small > n * hkv * D / 2


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D,group", [(64, 4), (128, 4), (128, 8), (128, 12)])
def test_paged_rows_not_finite(cuda_lib, dtype, wide, D, group):
    """NaN (and, in 16 bits, infinities) in single elements of values reach those elements of
    the output; in a key, the whole sequence; other sequences and kv heads are as ever."""
    lens, hkv = [700, 300, 90], 2

    def edit(k, v):
        v[5, 0, 3] = math.nan
        v[698, 0, 9] = math.nan if dtype == E4M3 else math.inf
        v[333, 1, D - 1] = math.nan
        k[700 + 260, 1, 2] = math.nan
        k[1000 + 89] = 0
    cache, table, _, _ = fill(cuda_lib, lens, 32, hkv, D, dtype, seed=31, edit=edit)
    q = normal(gen(32), 3, hkv * group, D)
    got = cuda_lib.paged_attention(q, cache, ints(lens),
                                   widened(table, 32, hkv) if wide else table)
    cuda_lib.sync_status()
    for s, n in enumerate(lens):
        k, v = rows_of(cache, table, s, n)
        for h in range(hkv * group):
            see = torch.ones((1, n), dtype=torch.bool, device=DEV)
            o, a = attend(q[s:s + 1, h], k[:, h // group], v[:, h // group], see, D ** -0.5)
            x, fin = got[s:s + 1, h].double(), torch.isfinite(o)
            assert torch.equal(torch.isnan(x), torch.isnan(o)), (s, h)
            assert torch.equal(x[torch.isinf(o)], o[torch.isinf(o)])
            close(torch.where(fin, x, 0.0), torch.where(fin, o, 0.0), torch.where(fin, a, 0.0))


# ------------------------------------------------------------------ beyond 32 bits
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
def test_cache_beyond_32_bits(cuda_lib, dtype, D):
    """A cache of more than 2^32 elements, whose last pages hold the sequences: written, read
    back and attended to."""
    page, hkv, group, lens = 128, 8, 2, [300, 5, 129]
    n_pages = 2 ** 32 // (page * hkv * D) + 8
    cache = cuda_lib.make_kv_cache(n_pages, page, hkv, D, dtype=dtype)
    small = cuda_lib.make_kv_cache(6, page, hkv, D, dtype=dtype)
    table = torch.tensor([[5, 0, 3], [1, -1, -1], [4, 2, -1]], dtype=torch.int32, device=DEV)
    far = torch.where(table >= 0, table + (n_pages - 6), table)
    g = gen(33)
    k, v = normal(g, sum(lens), hkv, D), normal(g, sum(lens), hkv, D)
    q = normal(g, 3, hkv * group, D)
    got = []
    for c, t in ((small, table), (cache, far)):
        cuda_lib.kv_cache_append(c, k, v, ints(lens), t, starts(lens))
        got.append([*cuda_lib.kv_cache_gather(c, t, starts(lens), total=sum(lens)),
                    cuda_lib.paged_attention(q, c, ints(lens), t),
                    cuda_lib.paged_attention(q, c, ints(lens), widened(t, page, hkv))])
    cuda_lib.sync_status()
    for a, b in zip(*got):
        assert torch.equal(a, b)
    o, a = attend_clean(q[0:1, 5], *(x[:, 2] for x in rows_of(small, table, 0, 300)),
                        torch.ones((1, 300), dtype=torch.bool, device=DEV), D ** -0.5)
    close(got[1][2][0:1, 5], o, a)


@pytest.mark.parametrize("causal", [True, False])
def test_packed_strides_beyond_32_bits(cuda_lib, causal):
    """Tokens 2^23 elements apart: the last ones lie behind 2^31 elements."""
    n, stride, D = 300, 2 ** 23, 64
    g = gen(34)
    dense = normal(g, n, 4, D)
    buf = torch.empty(n * stride, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((n, 8, D), (stride, D, 1))
    x[:, :4] = dense
    out = x[:, 4:6]
    want = cuda_lib.packed_attention(dense[:, :2], dense[:, 2:3], dense[:, 3:], starts([100, 200]),
                                     causal=causal)
    # (the output between the inputs' rows would be refused: it has a buffer of its own)
    out = torch.empty(n * stride // 4, dtype=torch.bfloat16, device=DEV).as_strided(
        (n, 2, D), (stride // 4, D, 1))
    cuda_lib.packed_attention(x[:, :2], x[:, 2:3], x[:, 3:4], starts([100, 200]), out=out,
                              causal=causal)
    cuda_lib.sync_status()
    assert torch.equal(out, want)


# ------------------------------------------------------------------ the rest
@pytest.mark.parametrize("D", [64, 128])
def test_packed_lowest_values_seen(cuda_lib, D):
    """Keys of the type's lowest value have scores of -inf: the rows that see them are those of
    the other keys."""
    n, ok = 300, 60
    g = gen(35)
    q, k, v = (normal(g, n, 1, D) for _ in range(3))
    q = q.abs()
    k[ok:] = torch.finfo(torch.bfloat16).min
    got = cuda_lib.packed_attention(q, k, v, starts([n]))
    cuda_lib.sync_status()
    see = causal_mask(n, n) & (torch.arange(n, device=DEV) < ok)[None]
    o, a = attend_clean(q[:, 0], k[:, 0], v[:, 0], see, D ** -0.5)
    close(got[:, 0], o, a)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C", [96, 1040, 4096])
def test_gated_norm_of_many_tokens(cuda_lib, dtype, C):
    """More rows than a wave of blocks holds: both outputs of every row (bounds as in
    test_gated_norm)."""
    g = gen(36)
    n = 20011 if C < 1000 else 7001
    x, f = normal(g, n, C, dtype=dtype), normal(g, n, C, dtype=dtype)
    gp, gn = (torch.rand(C, generator=g, device=DEV) + 0.5 for _ in range(2))
    gate = normal(g, -(-n // 700), C, dtype=torch.float32)
    y, m = cuda_lib.gated_residual_norm(x, f, gp, gate, gn, tokens_per_gate=700,
                                        residual_scale=0.6)
    cuda_lib.sync_status()
    u = U if dtype == torch.bfloat16 else 2.0 ** -24
    ry, rm, parts = norm_reference(x, f, gp, gate, 700, 0.6, gn, 1e-12)
    assert ((y.double() - ry).abs() <= u * ry.abs() + 2.0 ** -20 * parts).all()
    scale = C ** 0.5 / ry.norm(dim=-1, keepdim=True) * gn.double()
    assert ((m.double() - rm).abs() <= u * rm.abs() + 2.0 ** -19 * parts * scale.abs()).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C", [32, 384, 4096])
def test_gated_norm_rows_not_finite(cuda_lib, dtype, C):
    """A NaN in a row makes its norm NaN, and with it the whole normed row; an infinity makes
    it infinite: NaN where it lies, zeros elsewhere.  Other rows are as ever."""
    g = gen(37)
    n = 40
    x, f = normal(g, n, C, dtype=dtype), normal(g, n, C, dtype=dtype)
    gp, gn = (torch.rand(C, generator=g, device=DEV) + 0.5 for _ in range(2))
    f[3, 5], f[7, C - 1] = math.nan, math.inf
    x[11, 2], x[13, 9] = math.nan, -math.inf
    y, m = cuda_lib.gated_residual_norm(x, f, gp, None, gn)
    cuda_lib.sync_status()
    ry, rm, parts = norm_reference(x, f, gp, None, 1, 1.0, gn, 1e-12)
    u = U if dtype == torch.bfloat16 else 2.0 ** -24
    scale = C ** 0.5 / ry.norm(dim=-1, keepdim=True) * gn.double()
    for got, want, bar in ((y.double(), ry, u * ry.abs() + 2.0 ** -20 * parts),
                           (m.double(), rm, u * rm.abs() + 2.0 ** -19 * parts * scale.abs())):
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])
        fin = torch.isfinite(want) & torch.isfinite(bar)
        assert ((got - want).abs() <= bar)[fin].all()
        still = torch.ones(n, dtype=torch.bool, device=DEV)
        still[[3, 7, 11, 13]] = False
        assert fin[still].all()


@pytest.mark.parametrize("D,group", [(64, 4), (64, 12), (128, 2), (128, 8), (128, 12)])
@pytest.mark.parametrize("wide", [False, True])
def test_paged_bits_do_not_depend_on_the_call_before(cuda_lib, D, group, wide):
    """Short sequences leave most of a unit's places unread: what an earlier call left in
    shared memory there (scales of 2^-100, of 2^100) changes no bit of the result."""
    hkv, page = 8, 16
    lens = [(37 * i) % 200 for i in range(100)]
    cache, table, _, _ = fill(cuda_lib, lens, page, hkv, D, E4M3, seed=40)
    q = normal(gen(41), len(lens), hkv * group, D)
    if wide:
        table = widened(table, page, hkv)
    before = []
    for size in (2.0 ** -95, 2.0 ** 105):
        def edit(k, v):
            v *= size
            k *= 2.0 ** -10
        c, t, _, _ = fill(cuda_lib, [2000] * 20, page, hkv, D, E4M3, seed=42, edit=edit)
        if wide:
            t = widened(t, page, hkv)
        before.append((normal(gen(43), 20, hkv * group, D), c, ints([2000] * 20), t))
    got = []
    for args in (None, *before, *before):
        if args is not None:
            cuda_lib.paged_attention(*args)
        got.append(cuda_lib.paged_attention(q, cache, ints(lens), table))
    cuda_lib.sync_status()
    for a in got[1:]:
        assert torch.equal(got[0], a)
