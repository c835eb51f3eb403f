"""The sequence operators on the GPU: attention over packed sequences, the
paged key-value cache (written, read back, attended to) and the gated residual
with the norms around it, each against its definition in 64 bits.

Tolerances.  u = 2^-8 is half a step of bf16 relative to the value (the last
rounding of every bf16 output).  Attention also rounds its weights: p (1 + d) with
|d| <= u in bf16 (packed, and the bf16 cache) and below 2^-11 in fp16 (the 8-bit
cache), so an output o = sum p v / sum p moves by at most u * sum p |v| / sum p.
fp32 sums over n <= 2^13 keys add less than 2^-10 of the same magnitude (errors of
n random roundings of 2^-24, and scores that are off by D roundings, times a
score's size of at most 2^6).  With A = sum p |v| / sum p, the bound of an element is
u |o| + (u + 2^-10) A.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -8


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def starts(lens):
    return ints([sum(lens[:i]) for i in range(len(lens) + 1)])


def attend(q, k, v, see, scale):
    """64 bits: q [Lq, D], k and v [Lk, D], see [Lq, Lk] -> (o, sum p |v| / sum p);
    what is not seen takes no part."""
    q, k, v = q.double(), k.double(), v.double()
    o = torch.zeros((q.shape[0], v.shape[1]), dtype=torch.float64, device=q.device)
    a = torch.zeros_like(o)
    for i in range(q.shape[0]):
        at = see[i].nonzero()[:, 0]
        if at.numel():
            p = torch.softmax(k[at] @ q[i] * scale, 0)
            o[i], a[i] = p @ v[at], p @ v[at].abs()
    return o, a


def attend_clean(q, k, v, see, scale):
    """attend() for finite inputs, whole matrices at once."""
    s = (q.double() @ k.double().T * scale).masked_fill(~see, -math.inf)
    p = torch.softmax(s, 1)
    p = torch.where(see.any(1, keepdim=True), p, 0.0)
    return p @ v.double(), p @ v.double().abs()


def close(got, o, a, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    d = (got - o).abs()
    bar = U * o.abs() + (U + 2.0 ** -10) * a
    over = d - bar
    assert (over <= 0).all(), (
        f"{what}: off by {d.flatten()[over.argmax()].item():.3e}, "
        f"allowed {bar.flatten()[over.argmax()].item():.3e}")


def causal_mask(lq, lk):
    i, j = torch.arange(lq, device=DEV)[:, None], torch.arange(lk, device=DEV)[None]
    return j <= i + lk - lq


def packed_check(lib, lq, lk, hkv, group, D, causal, seed=0, scale=None, edit=None, ref=attend_clean,
                 behind=3, **kw):
    g = gen(seed)
    hq, Tq, Tk = hkv * group, sum(lq) + behind, sum(lk) + behind
    row = normal(g, Tq, (hq + 1) * D)          # strided queries
    q = row[:, :hq * D].view(Tq, hq, D) if group else None
    kv = normal(g, Tk, 2 * hkv, D)
    k, v = kv[:, :hkv], kv[:, hkv:]
    if edit:
        edit(q, k, v)
    out = torch.full((Tq, hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    got = lib.packed_attention(q, k, v, starts(lq), starts(lk), out=out, causal=causal,
                               scale=scale, **kw)
    lib.sync_status()
    assert torch.equal(got[sum(lq):], torch.full_like(got[sum(lq):], 7.0)), "rows behind the last"
    qa = ka = 0
    for n, m in zip(lq, lk):
        see = causal_mask(n, m) if causal else torch.ones((n, m), dtype=torch.bool, device=DEV)
        for h in range(hq):
            o, a = ref(q[qa:qa + n, h], k[ka:ka + m, h // group], v[ka:ka + m, h // group], see,
                       D ** -0.5 if scale is None else scale)
            close(got[qa:qa + n, h], o, a, f"{lq} {lk} head {h} at {qa}")
        qa, ka = qa + n, ka + m
    return got


# ------------------------------------------------------------------ packed attention
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", [[1], [127], [128], [129], [300, 1, 64], [0, 5, 0, 257, 0]])
def test_packed_self(cuda_lib, D, causal, lens):
    packed_check(cuda_lib, lens, lens, 2, 1, D, causal, seed=len(lens) + D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 16, 48, 128])
def test_packed_groups(cuda_lib, D, group):
    packed_check(cuda_lib, [37, 150], [37, 150], 1 if group > 8 else 2, group, D, True, seed=group)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_packed_other_lengths(cuda_lib, D, causal):
    # more keys than queries (new tokens of a longer sequence), fewer (queries
    # that see nothing), none at all
    packed_check(cuda_lib, [5, 200, 140, 9], [300, 130, 0, 9], 2, 2, D, causal, seed=3)


@pytest.mark.parametrize("D", [64, 128])
def test_packed_long(cuda_lib, D):
    packed_check(cuda_lib, [2500, 1111], [2500, 1111], 1, 2, D, True, seed=5)


@pytest.mark.parametrize("scale", [1e-4, 1.0, 4.0])
def test_packed_scales(cuda_lib, scale):
    # scores up to a few hundred: the running maximum moves, O is rescaled
    packed_check(cuda_lib, [700], [700], 1, 1, 64, True, seed=6, scale=scale)


def test_packed_rising_scores(cuda_lib):
    # every block's maximum far above the last one's: a rescale at every block
    def edit(q, k, v):
        q[:] = 1.0
        k[:] = torch.arange(k.shape[0], device=DEV)[:, None, None] / 16.0
    packed_check(cuda_lib, [900], [900], 1, 2, 128, True, seed=7, edit=edit)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_packed_other_sequences_do_not_leak(cuda_lib, causal, bad):
    # everything of the second sequence, and the rows behind the last, is not finite
    lens = [70, 40, 90]

    def edit(q, k, v):
        for t in (q, k, v):
            t[70:110] = bad
            t[200:] = bad
    g = gen(8)
    q, k, v = (normal(g, 203, 2, 64) for _ in range(3))
    edit(q, k, v)
    got = cuda_lib.packed_attention(q, k, v, starts(lens), causal=causal)
    cuda_lib.sync_status()
    for a, n in ((0, 70), (110, 90)):
        see = causal_mask(n, n) if causal else torch.ones((n, n), dtype=torch.bool, device=DEV)
        for h in range(2):
            o, m = attend_clean(q[a:a + n, h], k[a:a + n, h], v[a:a + n, h], see, 0.125)
            close(got[a:a + n, h], o, m, f"sequence at {a}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_packed_causal_future_does_not_leak(cuda_lib, D, bad):
    # the last keys and values of a sequence are not finite: queries before them are clean
    n, ok = 200, 150
    g = gen(9)
    q, k, v = (normal(g, n, 1, D) for _ in range(3))
    k[ok:] = bad
    v[ok:] = bad
    got = cuda_lib.packed_attention(q, k, v, starts([n]))
    cuda_lib.sync_status()
    o, a = attend_clean(q[:ok, 0], k[:ok, 0], v[:ok, 0], causal_mask(ok, ok), D ** -0.5)
    close(got[:ok, 0], o, a, "before the first bad key")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 8])
def test_packed_causal_values_not_finite(cuda_lib, D, group):
    # infinities and NaN in single elements of values: the rows that see them, and no
    # others, get them (of both signs: NaN), in those elements alone
    n, hkv = 430, 2
    g = gen(13)
    q, k, v = (normal(g, n, h, D) for h in (hkv * group, hkv, hkv))
    v[5, 0, 3] = math.inf
    v[140, 0, 7], v[141, 0, 7], v[140, 0, 40] = math.inf, -math.inf, -math.inf
    v[129, 1, D - 1] = math.nan
    v[255:258, 1, 16] = -math.inf
    v[n - 1, 0] = math.nan
    v[n - 2, 1, 0] = math.inf
    got = cuda_lib.packed_attention(q, k, v, starts([n]))
    cuda_lib.sync_status()
    for h in range(hkv * group):
        o, a = attend(q[:, h], k[:, h // group], v[:, h // group], causal_mask(n, n), D ** -0.5)
        x, fin = got[:, h].double(), torch.isfinite(o)
        assert torch.equal(torch.isnan(x), torch.isnan(o))
        assert torch.equal(x[torch.isinf(o)], o[torch.isinf(o)])
        close(torch.where(fin, x, 0.0), torch.where(fin, o, 0.0), torch.where(fin, a, 0.0))


@pytest.mark.parametrize("causal", [True, False])
def test_packed_values_all_nan(cuda_lib, causal):
    # every value is NaN: every row that sees a key is NaN, one that sees none is zero
    g = gen(14)
    q, k = normal(g, 300, 4, 64), normal(g, 260, 1, 64)
    v = torch.full_like(k, math.nan)
    got = cuda_lib.packed_attention(q, k, v, starts([300]), starts([260]), causal=causal)
    cuda_lib.sync_status()
    first = 40 if causal else 0
    assert torch.isnan(got[first:]).all() and (got[:first] == 0).all()


def test_packed_lowest_value_rows(cuda_lib):
    # keys of the type's lowest value give scores of -inf and +inf's neighbours
    # where they are seen, and nothing where they are masked
    n = 100
    g = gen(10)
    q, k, v = (normal(g, n, 1, 64) for _ in range(3))
    q = q.abs()
    k[60:] = torch.finfo(torch.bfloat16).min
    got = cuda_lib.packed_attention(q, k, v, starts([n]))
    cuda_lib.sync_status()
    o, a = attend_clean(q[:60, 0], k[:60, 0], v[:60, 0], causal_mask(60, 60), 0.125)
    close(got[:60, 0], o, a)


def test_packed_bad_offsets_are_skipped(cuda_lib):
    g = gen(11)
    q, k, v = (normal(g, 100, 1, 64) for _ in range(3))
    cu = ints([0, 40, 120])
    out = torch.full_like(q, 7.0)
    cuda_lib.packed_attention(q, k, v, cu, out=out)
    with pytest.raises(cuda_lib.WanvaeError) as ei:
        cuda_lib.sync_status()
    assert ei.value.status == cuda_lib.ERR_CUDA
    o, a = attend_clean(q[:40, 0], k[:40, 0], v[:40, 0], causal_mask(40, 40), 0.125)
    close(out[:40, 0], o, a)
    assert torch.all(out[40:] == 7.0)


def test_packed_timeout_reports_and_context_survives(cuda_lib):
    g = gen(12)
    q, k, v = (normal(g, 300, 2, 128) for _ in range(3))
    cu = starts([300])
    cuda_lib.sync_status()
    try:
        cuda_lib.set_wait_limit_ns(0)
        cuda_lib.packed_attention(q, k, v, cu)
        with pytest.raises(cuda_lib.WanvaeError) as ei:
            cuda_lib.sync_status()
        assert ei.value.status == cuda_lib.ERR_TIMEOUT
    finally:
        cuda_lib.set_wait_limit_ns(10 ** 9)
    got = cuda_lib.packed_attention(q, k, v, cu)
    cuda_lib.sync_status()
    o, a = attend_clean(q[:, 1], k[:, 1], v[:, 1], causal_mask(300, 300), 128 ** -0.5)
    close(got[:, 1], o, a)


def test_packed_graph_and_other_stream(cuda_lib):
    g = gen(15)
    qkv = normal(g, 400, 6, 128)
    cu = starts([150, 250])
    want = cuda_lib.packed_attention(qkv[:, :4], qkv[:, 4:5], qkv[:, 5:], cu)
    cuda_lib.sync_status()
    src, out = torch.zeros_like(qkv), torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        cuda_lib.packed_attention(src[:, :4], src[:, 4:5], src[:, 5:], cu, out=out)
        y, _ = cuda_lib.gated_residual_norm(out, want)
    src.copy_(qkv)
    graph.replay()
    torch.cuda.synchronize()
    cuda_lib.sync_status()
    assert torch.equal(out, want) and torch.equal(y, want + want)
    got = cuda_lib.packed_attention(qkv[:, :4], qkv[:, 4:5], qkv[:, 5:], cu, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


# ------------------------------------------------------------------ the cache
def quantised(x):
    """The definition in 64 bits: (values of the elements, exponents)."""
    x = x.double()
    fin = torch.where(torch.isfinite(x), x, 0.0)
    amax = fin.abs().amax(-1)
    m, e = torch.frexp(amax / 448.0)
    e = torch.where(m == 0.5, e - 1, e).clamp(-100, 120)
    e = torch.where(amax == 0, 0, e)
    two = lambda n: ((n.long() + 1023) << 52).view(torch.float64)  # noqa: E731
    z = fin / two(e)[..., None]
    step = two((torch.frexp(z)[1] - 1).clamp_min(-6) - 3)
    z = torch.round(z / step) * step
    return torch.where(torch.isfinite(x), z, math.nan), e


def table_for(lens, page, seed=0, spare=2):
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=torch.Generator().manual_seed(seed)).tolist()
    t = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    for s, n in enumerate(need):
        t[s, :n] = torch.tensor(order[:n], dtype=torch.int32)
        order = order[n:]
    return t.to(DEV), sum(need) + spare


def rows_of(cache, table, s, n):
    """The cache's key and value rows (64 bits) of positions 0 .. n - 1 of sequence s."""
    got = []
    pos = torch.arange(n, device=DEV)
    page = table[s].long()[pos // cache.page_size]
    for x, e in ((cache.k, cache.k_exp), (cache.v, cache.v_exp)):
        if e is None:
            got.append(x[page, :, pos % cache.page_size].double())
        else:
            r = x.view(torch.uint8)[page, :, pos % cache.page_size].view(torch.float8_e4m3fn)
            c = e.view(torch.uint8)[page, :, pos % cache.page_size].long() - 127
            got.append(r.double() * ((c + 1023) << 52).view(torch.float64)[..., None])
    return got


def fill(lib, lens, page, hkv, D, dtype, seed=0, edit=None):
    """A cache written through the library, and its page table."""
    g = gen(seed)
    table, n_pages = table_for(lens, page, seed)
    cache = lib.make_kv_cache(n_pages, page, hkv, D, dtype=dtype)
    k = normal(g, sum(lens), hkv, D) * torch.exp(normal(g, sum(lens), hkv, 1))
    v = normal(g, sum(lens), hkv, D) * torch.exp(normal(g, sum(lens), hkv, 1))
    if edit:
        edit(k, v)
    if sum(lens):
        lib.kv_cache_append(cache, k, v, ints(lens), table, starts(lens))
    return cache, table, k, v


DTYPES = [torch.float8_e4m3fn, torch.bfloat16]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hkv", [1, 3, 8])
@pytest.mark.parametrize("page", [16, 128])
def test_cache_append(cuda_lib, dtype, D, hkv, page):
    lens = [1, 40, 0, 129]
    cache, table, k, v = fill(cuda_lib, lens, page, hkv, D, dtype, seed=hkv)
    cuda_lib.sync_status()
    at = 0
    for s, n in enumerate(lens):
        for x, got in zip((k, v), rows_of(cache, table, s, n)):
            x = x[at:at + n]
            if dtype == torch.bfloat16:
                want = x.double()
            else:
                z, e = quantised(x)
                want = z * torch.exp2(e.double())[..., None]
            assert torch.equal(got, want)
        at += n


@pytest.mark.parametrize("D", [64, 128])
def test_cache_append_extremes(cuda_lib, D):
    # zeros, the borders of a scale, denormals, the largest values, not finite ones
    big = torch.finfo(torch.bfloat16).max
    rows = [0.0, 448.0, 450.0, 447.0, 1.0, 2.0 ** -130, 2.0 ** -109, 2.0 ** -92, big, -big, 7.0, 3.5]
    x = torch.zeros((len(rows) + 3, 1, D), dtype=torch.bfloat16, device=DEV)
    for i, r in enumerate(rows):
        x[i, 0] = torch.linspace(-1, 1, D, device=DEV) * 0.9 * r
        x[i, 0, i] = r
    x[-3] = torch.linspace(-2, 2, D, device=DEV)
    x[-3, 0, 0], x[-3, 0, 1] = math.inf, math.nan
    x[-2] = -math.inf
    x[-1] = math.nan
    n = x.shape[0]
    cache = cuda_lib.make_kv_cache(1, 32, 1, D)
    cuda_lib.kv_cache_append(cache, x, -x, ints([n]), ints([[0]]), starts([n]))
    cuda_lib.sync_status()
    z, e = quantised(x)
    for sign, t, c in ((1, cache.k, cache.k_exp), (-1, cache.v, cache.v_exp)):
        got = t[0, 0, :n].double()
        assert torch.equal(torch.isnan(got), torch.isnan(z[:, 0]))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(sign * z[:, 0]))
        assert torch.equal(c.view(torch.uint8)[0, 0, :n].long() - 127, e[:, 0].long())


def test_cache_append_step_by_step_equals_at_once(cuda_lib):
    lens, page, hkv, D = [33, 7, 64], 16, 2, 128
    whole, table, k, v = fill(cuda_lib, lens, page, hkv, D, torch.float8_e4m3fn, seed=1)
    steps = cuda_lib.make_kv_cache(whole.k.shape[0], page, hkv, D)
    first = [0, 33, 40]
    for i in range(max(lens)):
        on = [s for s in range(3) if i < lens[s]]
        rows = torch.tensor([first[s] + i for s in on], device=DEV)
        cuda_lib.kv_cache_append(steps, k[rows], v[rows], ints([i + 1] * len(on)),
                                 table[on].contiguous())
    cuda_lib.sync_status()
    for a, b in zip(whole.tensors(), steps.tensors()):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_cache_gather(cuda_lib, dtype, D, hkv):
    lens = [1, 300, 0, 77, 16]
    cache, table, _, _ = fill(cuda_lib, lens, 32, hkv, D, dtype, seed=D)
    T = sum(lens)
    both = torch.full((T + 2, 2 * hkv, D), 7.0, dtype=torch.bfloat16, device=DEV)
    k, v = cuda_lib.kv_cache_gather(cache, table, starts(lens), k=both[:, :hkv], v=both[:, hkv:])
    cuda_lib.sync_status()
    at = 0
    for s, n in enumerate(lens):
        for got, want in zip((k, v), rows_of(cache, table, s, n)):
            assert torch.equal(got[at:at + n].double(), want)  # e4m3 * 2^e is a bf16 value
        at += n
    assert torch.all(both[T:] == 7.0)


def test_cache_bad_pages_are_left_out(cuda_lib):
    lens, page = [40], 16
    cache = cuda_lib.make_kv_cache(4, page, 1, 64)
    before = [t.view(torch.uint8).clone() for t in cache.tensors()]
    g = gen(2)
    k, v = normal(g, 40, 1, 64), normal(g, 40, 1, 64)
    table = ints([[1, 9, -1]])
    cuda_lib.kv_cache_append(cache, k, v, ints(lens), table, starts(lens))
    with pytest.raises(cuda_lib.WanvaeError):
        cuda_lib.sync_status()
    for t, b in zip(cache.tensors(), before):
        keep = [0, 2, 3]
        assert torch.equal(t.view(torch.uint8)[keep], b[keep])
    out = torch.full((40, 1, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    cuda_lib.kv_cache_gather(cache, table, starts(lens), k=out, v=out.clone())
    with pytest.raises(cuda_lib.WanvaeError):
        cuda_lib.sync_status()
    assert torch.all(out[16:] == 7.0)
    # a length beyond the page table: positions outside are not written
    cuda_lib.kv_cache_append(cache, k[:2], v[:2], ints([49]), ints([[0, 1, 2]]), starts([2]))
    with pytest.raises(cuda_lib.WanvaeError):
        cuda_lib.sync_status()
    q = normal(g, 1, 2, 64)
    cuda_lib.paged_attention(q, cache, ints([40]), table)
    with pytest.raises(cuda_lib.WanvaeError):
        cuda_lib.sync_status()
    cuda_lib.paged_attention(q, cache, ints([60]), ints([[0, 1, 2]]))
    with pytest.raises(cuda_lib.WanvaeError):
        cuda_lib.sync_status()
    cuda_lib.sync_status()


# ------------------------------------------------------------------ one token over the cache
# What a call runs depends on how far its page table reaches: 8-bit caches of 128-element
# heads behind long tables have a kernel of their own.
def widened(table, page, hkv):
    """The table, reaching 2^18 rows over all sequences and kv heads and 4096 in each."""
    reach = max(4096, -(-2 ** 18 // (table.shape[0] * hkv)))
    out = torch.full((table.shape[0], -(-reach // page)), -1, dtype=torch.int32, device=DEV)
    out[:, :table.shape[1]] = table[:, :out.shape[1]]
    return out if out.shape[1] > table.shape[1] else table


def paged_check(lib, lens, page, hkv, group, D, dtype, seed=0, scale=None, edit=None, **kw):
    cache, narrow, _, _ = fill(lib, lens, page, hkv, D, dtype, seed, edit)
    g = gen(seed + 100)
    row = normal(g, len(lens), hkv * group + 1, D)
    q = row[:, :hkv * group]
    for table in (narrow, widened(narrow, page, hkv)):
        got = lib.paged_attention(q, cache, ints(lens), table, scale=scale, **kw)
        lib.sync_status()
        for s, n in enumerate(lens):
            k, v = rows_of(cache, narrow, s, n)
            see = torch.ones((1, n), dtype=torch.bool, device=DEV)
            for h in range(hkv * group):
                o, a = attend_clean(q[s:s + 1, h], k[:, h // group], v[:, h // group], see,
                                    D ** -0.5 if scale is None else scale)
                close(got[s:s + 1, h], o, a, f"sequence {s} of {n}, head {h}")
    return got


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [1, 3, 8, 9, 16, 20])
def test_paged_groups(cuda_lib, dtype, D, group):
    paged_check(cuda_lib, [5, 300, 64], 16, 2, group, D, dtype, seed=group)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[1], [0], [0, 17, 0, 0, 65, 0], [63], [64], [129],
                                  [1, 2, 3, 4, 5, 6, 7] * 10])
def test_paged_lengths(cuda_lib, dtype, lens):
    paged_check(cuda_lib, lens, 32, 2, 4, 128, dtype, seed=len(lens))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [16, 64, 1024])
def test_paged_long_and_ragged(cuda_lib, dtype, page):
    paged_check(cuda_lib, [4111, 9, 0, 8192, 700], page, 1, 4, 128, dtype, seed=page)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [1e-4, 1.0, 3.0])
def test_paged_scales(cuda_lib, dtype, scale):
    paged_check(cuda_lib, [2000, 90], 64, 1, 8, 64, dtype, seed=4, scale=scale)


def test_paged_value_scales_far_apart(cuda_lib):
    # rows of values from 2^-90 to 2^90 of each other, and a query of tiny elements
    def edit(k, v):
        v *= torch.exp2(torch.linspace(-60, 60, v.shape[0], device=DEV))[:, None, None]
    paged_check(cuda_lib, [500], 16, 1, 4, 64, torch.float8_e4m3fn, seed=5, edit=edit)

    def back(k, v):
        edit(k, v)
        v[:] = v.flip(0)
    paged_check(cuda_lib, [500], 16, 1, 4, 64, torch.float8_e4m3fn, seed=6, edit=back)


def test_paged_behind_the_length_does_not_leak(cuda_lib):
    lens, D = [21, 75], 64
    cache, table, _, _ = fill(cuda_lib, [32, 80], 16, 1, D, torch.bfloat16, seed=7)
    for s, n in enumerate(lens):
        for p in range(n, [32, 80][s]):
            cache.k[table[s, p // 16], :, p % 16] = math.nan
            cache.v[table[s, p // 16], :, p % 16] = math.inf
    q = normal(gen(8), 2, 2, D)
    got = cuda_lib.paged_attention(q, cache, ints(lens), table)
    cuda_lib.sync_status()
    for s, n in enumerate(lens):
        k, v = rows_of(cache, table, s, n)
        for h in range(2):
            o, a = attend_clean(q[s:s + 1, h], k[:, 0], v[:, 0],
                                torch.ones((1, n), dtype=torch.bool, device=DEV), 0.125)
            close(got[s:s + 1, h], o, a)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [16, 32, 128, 256, 1024])
def test_paged_behind_the_length_and_bad_pages(cuda_lib, dtype, page, wide):
    """D = 128: what lies behind the length is not finite (scales too); then a page that
    is not there, a negative length and one beyond the page table: the rest is attended."""
    full, lens, D, group = [2 * page, 1040 + page, 5 * page], [page + 3, 1037, 4 * page + 1], 128, 4
    cache, table, _, _ = fill(cuda_lib, full, page, 1, D, dtype, seed=page)
    kept = [rows_of(cache, table, s, n) for s, n in enumerate(full)]
    if wide:
        table = widened(table, page, 1)
    for s, n in enumerate(lens):
        pos = torch.arange(n, full[s], device=DEV)
        at = table[s].long()[pos // page]
        for x, bad in ((cache.k, math.nan), (cache.v, math.nan)):
            if dtype == torch.bfloat16:
                x[at, :, pos % page] = bad
            else:
                x.view(torch.uint8)[at, :, pos % page] = 0x7f
        for e in (cache.k_exp, cache.v_exp):
            if e is not None:
                e.view(torch.uint8)[at, :, pos % page] = 255
    q = normal(gen(9), 3, group, D)

    def check(got, seen):
        for s, (k, v) in enumerate(kept):
            see = torch.zeros((1, k.shape[0]), dtype=torch.bool, device=DEV)
            see[0, seen[s]] = True
            for h in range(group):
                o, a = attend(q[s:s + 1, h], k[:, 0], v[:, 0], see, D ** -0.5)
                close(got[s:s + 1, h], o, a, f"sequence {s}, head {h}")
    got = cuda_lib.paged_attention(q, cache, ints(lens), table)
    cuda_lib.sync_status()
    check(got, [torch.arange(n, device=DEV) for n in lens])
    broken = table.clone()
    broken[0, 0] = -1
    broken[2, 1] = cache.k.shape[0]
    got = cuda_lib.paged_attention(q, cache, ints([lens[0], -5, lens[2]]), broken)
    with pytest.raises(cuda_lib.WanvaeError):
        cuda_lib.sync_status()
    rest = torch.arange(lens[2], device=DEV)
    check(got, [torch.arange(page, lens[0], device=DEV), torch.arange(0, device=DEV),
                rest[rest // page != 1]])
    if wide:
        return  # a length beyond a table this long would be over pages that are not there
    narrow = table[:, :1].contiguous()
    got = cuda_lib.paged_attention(q, cache, ints([page, page + 1, 2 ** 31 - 1]), narrow)
    with pytest.raises(cuda_lib.WanvaeError):
        cuda_lib.sync_status()
    check(got, [torch.arange(page, device=DEV)] * 3)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [33, 700])
def test_paged_many_sequences_share_pages(cuda_lib, dtype, D, n):
    """Many short sequences, all of them over the same pages: more items than CTAs."""
    page, group = 16, 2
    cache, table, _, _ = fill(cuda_lib, [70], page, 2, D, dtype, seed=n)
    lens = [(7 * i) % 71 for i in range(n)]
    q = normal(gen(n), n, 2 * group, D)
    k, v = rows_of(cache, table, 0, 70)
    see = torch.arange(70, device=DEV)[None] < torch.tensor(lens, device=DEV)[:, None]
    shared = table.expand(n, -1).contiguous()
    for t in (shared, widened(shared, page, 2)):
        got = cuda_lib.paged_attention(q, cache, ints(lens), t)
        cuda_lib.sync_status()
        for h in range(2 * group):
            o, a = attend_clean(q[:, h], k[:, h // group], v[:, h // group], see, D ** -0.5)
            close(got[:, h], o, a, f"head {h}")
    kk, vv = cuda_lib.kv_cache_gather(cache, table.expand(n, -1).contiguous(), starts(lens),
                                      total=sum(lens))
    cuda_lib.sync_status()
    at = torch.cat([torch.arange(x, device=DEV) for x in lens])
    assert torch.equal(kk.double(), k[at]) and torch.equal(vv.double(), v[at])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("wide", [False, True])
def test_paged_query_not_finite(cuda_lib, dtype, bad, wide):
    """One head's query is not finite: that head's row is NaN, no other's."""
    cache, table, _, _ = fill(cuda_lib, [300, 40], 32, 2, 128, dtype, seed=4)
    if wide:
        table = widened(table, 32, 2)
    q = normal(gen(5), 2, 8, 128)
    clean = cuda_lib.paged_attention(q, cache, ints([300, 40]), table)
    q[0, 3, 17] = bad
    got = cuda_lib.paged_attention(q, cache, ints([300, 40]), table)
    cuda_lib.sync_status()
    assert torch.isnan(got[0, 3]).all()
    keep = torch.ones((2, 8), dtype=torch.bool, device=DEV)
    keep[0, 3] = False
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("dtype,D,wide", [
    (torch.float8_e4m3fn, 128, False), (torch.float8_e4m3fn, 128, True),
    (torch.float8_e4m3fn, 64, False), (torch.bfloat16, 128, False)])
def test_paged_timeout_reports_and_context_survives(cuda_lib, dtype, D, wide):
    lens = [3000, 17, 600]
    cache, table, _, _ = fill(cuda_lib, lens, 64, 2, D, dtype, seed=6)
    if wide:
        table = widened(table, 64, 2)
    q = normal(gen(6), 3, 8, D)
    want = cuda_lib.paged_attention(q, cache, ints(lens), table)
    cuda_lib.sync_status()
    try:
        cuda_lib.set_wait_limit_ns(0)
        cuda_lib.paged_attention(q, cache, ints(lens), table)
        with pytest.raises(cuda_lib.WanvaeError) as ei:
            cuda_lib.sync_status()
        assert ei.value.status == cuda_lib.ERR_TIMEOUT
    finally:
        cuda_lib.set_wait_limit_ns(10 ** 9)
    got = cuda_lib.paged_attention(q, cache, ints(lens), table)
    cuda_lib.sync_status()
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_paged_two_streams_at_once(cuda_lib, dtype):
    """Two calls at once, each with its own workspace, and a graph of each replayed on
    two streams: the results of calls one after another."""
    lens = [9000, 4000, 30]
    cache, table, _, _ = fill(cuda_lib, lens, 64, 2, 128, dtype, seed=8)
    table = widened(table, 64, 2)
    qs = [normal(gen(i), 3, 8, 128) for i in range(2)]
    at = [ints(lens), ints([n // 2 for n in lens])]
    want = [cuda_lib.paged_attention(qs[i], cache, at[i], table) for i in range(2)]
    outs = [torch.empty_like(w) for w in want]
    ws = [cuda_lib.make_paged_attention_workspace(qs[i], cache) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            cuda_lib.paged_attention(qs[i], cache, at[i], table, out=outs[i], workspace=ws[i])
    for eager in (True, False):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            for i in range(2):
                if eager:
                    cuda_lib.paged_attention(qs[i], cache, at[i], table, out=outs[i],
                                             workspace=ws[i], stream=streams[i])
                else:
                    with torch.cuda.stream(streams[i]):
                        graphs[i].replay()
        torch.cuda.synchronize()
        cuda_lib.sync_status()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


# ------------------------------------------------------------------ gated residual and norms
def norm_reference(x, f, gp, gate, per, s, gn, eps):
    """64 bits: y, and the norm of the unrounded y."""
    x, f = x.double(), f.double()
    C = x.shape[-1]

    def rms(t, gamma):
        return t / t.square().sum(-1, keepdim=True).sqrt().clamp_min(eps) * C ** 0.5 * gamma.double()
    h = rms(f, gp) if gp is not None else f
    if gate is not None:
        h = h * gate.double()[torch.arange(x.shape[0], device=DEV) // per]
    y = x + s * h
    return y, (rms(y, gn) if gn is not None else None), x.abs() + (s * h).abs()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C", [16, 48, 96, 112, 384, 1040, 2064, 4080, 4096])
@pytest.mark.parametrize("n", [1, 37])
def test_gated_norm(cuda_lib, dtype, C, n):
    """y within half a step of its type plus 2^-20 of what it was summed from;
    n likewise (fp32 sums of C <= 4096 squares are exact to 2^-20 here, and a
    channel where y cancels carries the error of its terms)."""
    g = gen(C + n)
    x, f = normal(g, n, C, dtype=dtype), normal(g, n, C, dtype=dtype)
    gp, gn = (torch.rand(C, generator=g, device=DEV) + 0.5 for _ in range(2))
    u = U if dtype == torch.bfloat16 else 2.0 ** -24
    for per, post, gated, pre in ((1, True, True, True), (5, True, True, True),
                                  (1, False, True, True), (1, True, False, True),
                                  (1, True, True, False), (1, False, False, False)):
        gate = normal(g, -(-n // per), C, dtype=torch.float32) if gated else None
        y, m = cuda_lib.gated_residual_norm(x, f, gp if post else None, gate, gn if pre else None,
                                            tokens_per_gate=per, residual_scale=0.6)
        cuda_lib.sync_status()
        ry, rm, parts = norm_reference(x, f, gp if post else None, gate, per, 0.6,
                                       gn if pre else None, 1e-12)
        assert ((y.double() - ry).abs() <= u * ry.abs() + 2.0 ** -20 * parts).all()
        if not pre:
            assert m is None
            continue
        scale = C ** 0.5 / ry.norm(dim=-1, keepdim=True) * gn.double()
        assert ((m.double() - rm).abs() <= u * rm.abs() + 2.0 ** -19 * parts * scale.abs()).all()


def test_gated_norm_zero_rows_and_many_tokens(cuda_lib):
    g = gen(1)
    n, C = 20011, 96
    x, f = normal(g, n, C), normal(g, n, C)
    x[5], f[5] = 0, 0
    gp, gn = (torch.rand(C, generator=g, device=DEV) + 0.5 for _ in range(2))
    gate = normal(g, 3, C, dtype=torch.float32)
    y, m = cuda_lib.gated_residual_norm(x, f, gp, gate, gn, tokens_per_gate=7000)
    cuda_lib.sync_status()
    assert torch.all(y[5] == 0) and torch.all(m[5] == 0)
    ry, rm, parts = norm_reference(x, f, gp, gate, 7000, 1.0, gn, 1e-12)
    assert ((y.double() - ry).abs() <= U * ry.abs() + 2.0 ** -20 * parts).all()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("D,hkv,group", [(64, 2, 3), (128, 1, 4)])
def test_whole_clip_and_token_by_token_agree(cuda_lib, D, hkv, group):
    """A causal block over a clip at once, and token by token over the cache
    (append, attend), with the norms and the gate around it: the bf16 cache holds
    the same keys and values, so the two agree to the roundings of both."""
    lens, C = [70, 33], hkv * group * D
    g = gen(20)
    T = sum(lens)
    x = normal(g, T, C)
    wqkv = (normal(g, C, (group + 2) * hkv * D, dtype=torch.float32) * C ** -0.5).bfloat16()
    wo = (normal(g, C, C, dtype=torch.float32) * C ** -0.5).bfloat16()
    gp, gn = (torch.rand(C, generator=g, device=DEV) + 0.5 for _ in range(2))
    gate = normal(g, 1, C, dtype=torch.float32)
    h = hkv * group

    def after(xs, o):
        return cuda_lib.gated_residual_norm(xs, (o.flatten(1) @ wo), gp, gate, gn,
                                            tokens_per_gate=1 << 20, residual_scale=0.7)

    qkv = (x @ wqkv).view(T, h + 2 * hkv, D)
    o = cuda_lib.packed_attention(qkv[:, :h], qkv[:, h:h + hkv], qkv[:, h + hkv:], starts(lens))
    y, n = after(x, o)
    table, n_pages = table_for(lens, 16)
    cache = cuda_lib.make_kv_cache(n_pages, 16, hkv, D, dtype=torch.bfloat16)
    first = [0, lens[0]]
    for i in range(max(lens)):
        on = [s for s in range(2) if i < lens[s]]
        rows = torch.tensor([first[s] + i for s in on], device=DEV)
        t, at = table[on].contiguous(), ints([i + 1] * len(on))
        step = qkv[rows]
        cuda_lib.kv_cache_append(cache, step[:, h:h + hkv], step[:, h + hkv:], at, t)
        one = cuda_lib.paged_attention(step[:, :h], cache, at, t)
        # both are within 2 u + 2^-10 of sum p |v| / sum p <= max |v| of the exact value
        bar = 2 * (2 * U + 2.0 ** -10) * qkv[:, h + hkv:].abs().max()
        assert ((one.double() - o[rows].double()).abs() <= bar).all()
        y1, n1 = after(x[rows], one)
        assert torch.isfinite(n1.float()).all() and y1.shape == y[rows].shape
    cuda_lib.sync_status()
    # a pass over the last tokens alone, over the cache read back
    new = [20, 5]
    kb, vb = cuda_lib.kv_cache_gather(cache, table, starts(lens), total=T)
    at = torch.cat([torch.arange(first[s] + lens[s] - new[s], first[s] + lens[s]) for s in (0, 1)])
    part = cuda_lib.packed_attention(qkv[at.to(DEV), :h], kb, vb, starts(new), starts(lens))
    cuda_lib.sync_status()
    assert ((part.double() - o[at.to(DEV)].double()).abs() <= bar).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_graph_replay_and_other_stream(cuda_lib, dtype):
    """One decoding step captured once and replayed with new inputs in the same
    tensors, on a stream of its own, gives the eager calls' bits."""
    lens, hkv, group, D = [50, 200], 2, 2, 64
    cache, table, _, _ = fill(cuda_lib, [52, 202], 16, hkv, D, dtype, seed=3)
    g = gen(9)
    q = normal(g, 2, hkv * group, D)
    k, v = normal(g, 2, hkv, D), normal(g, 2, hkv, D)
    at, out = ints([n + 1 for n in lens]), torch.empty_like(q)
    ws = cuda_lib.make_paged_attention_workspace(q, cache)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        cuda_lib.kv_cache_append(cache, k, v, at, table)
        cuda_lib.paged_attention(q, cache, at, table, out=out, workspace=ws)
    for step in range(2):
        q.copy_(normal(g, *q.shape))
        k.copy_(normal(g, *k.shape))
        at.fill_(51 + step)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = cuda_lib.paged_attention(q, cache, at, table)
        cuda_lib.sync_status()
        assert torch.equal(got, want)


def test_runs_repeat_bit_for_bit(cuda_lib):
    cache, table, _, _ = fill(cuda_lib, [3000, 40, 555], 64, 2, 128, torch.float8_e4m3fn, seed=2)
    g = gen(4)
    q = normal(g, 3, 8, 128)
    a = [cuda_lib.paged_attention(q, cache, ints([3000, 40, 555]), table) for _ in range(3)]
    wide = widened(table, 64, 2)
    c = [cuda_lib.paged_attention(q, cache, ints([3000, 40, 555]), wide) for _ in range(3)]
    qkv = normal(g, 900, 6, 128)
    b = [cuda_lib.packed_attention(qkv[:, :4], qkv[:, 4:5], qkv[:, 5:], starts([500, 400]))
         for _ in range(3)]
    cuda_lib.sync_status()
    for runs in (a, b, c):
        assert all(torch.equal(runs[0], t) for t in runs)
