"""The sequence operators' calls: what they report, where their results are allocated, what
they refuse.  References and bounds as in test_seq_gpu.py."""
import pytest
import torch

from test_seq_gpu import DEV, attend_clean, causal_mask, close, gen, ints, normal, starts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,bad", [
    ([40] * 70, 35), ([40] * 70, 69), ([40] * 70, 0), ([0] * 50 + [300] + [0] * 40, 60),
    ([0] * 40 + [5], 33), ([1000] + [3] * 40, 38)])
@pytest.mark.parametrize("where", ["q", "k"])
def test_packed_bad_offsets_are_reported_wherever_they_are(cuda_lib, lens, bad, where):
    """One sequence's end lies outside the tensors, among more sequences than a warp looks at
    together: that sequence and the next (which begins there) are left out and reported, the
    others are computed."""
    g = gen(len(lens) + bad)
    T, out_of = sum(lens), 10 ** 6
    q, k, v = normal(g, T, 2, 64), normal(g, T, 1, 64), normal(g, T, 1, 64)
    cu = starts(lens)
    broken = cu.clone()
    broken[bad + 1] = out_of
    out = torch.full_like(q, 7.0)
    cuda_lib.packed_attention(q, k, v, broken if where == "q" else cu,
                              broken if where == "k" else cu, out=out)
    with pytest.raises(cuda_lib.WanvaeError) as ei:
        cuda_lib.sync_status()
    assert ei.value.status == cuda_lib.ERR_CUDA
    cuda_lib.sync_status()  # reported once
    at = 0
    for s, n in enumerate(lens):
        if s in (bad, bad + 1):
            assert torch.all(out[at:at + n] == 7.0)
        elif n:
            for h in range(2):
                o, a = attend_clean(q[at:at + n, h], k[at:at + n, 0], v[at:at + n, 0],
                                    causal_mask(n, n), 0.125)
                close(out[at:at + n, h], o, a, f"sequence {s}")
        at += n


def pool_of(t):
    """The stream whose memory a tensor lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


@pytest.mark.parametrize("what", ["packed", "gather", "paged", "norm"])
def test_results_lie_in_the_memory_of_the_call_s_stream(cuda_lib, what, monkeypatch):
    """With stream= and no outputs given, what the call allocates belongs to that stream: a
    block out of the current stream's memory may still be in use there.  (The streams
    are idle here: nothing overlaps.)"""
    g = gen(1)
    x = normal(g, 48, 2, 64)
    cache = cuda_lib.make_kv_cache(3, 16, 2, 64)
    table, lens, cu = ints([[0, 1, 2]]), ints([48]), ints([0, 48])
    cuda_lib.kv_cache_append(cache, x, x, lens, table, cu)
    made = []
    real = cuda_lib.make_paged_attention_workspace

    def workspace(*args):
        made.append(real(*args))
        return made[-1]
    monkeypatch.setattr(cuda_lib, "make_paged_attention_workspace", workspace)

    def call(stream):
        if what == "packed":
            return [cuda_lib.packed_attention(x, x, x, cu, stream=stream)]
        if what == "gather":
            return list(cuda_lib.kv_cache_gather(cache, table, cu, total=48, stream=stream))
        if what == "paged":
            return [cuda_lib.paged_attention(x[:1], cache, lens, table, stream=stream)]
        ones = torch.ones(64, device=DEV)
        return list(cuda_lib.gated_residual_norm(x, x, ones, None, ones, stream=stream))
    torch.cuda.synchronize()
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(side)
    side.synchronize()
    cuda_lib.sync_status()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    for t in got + made[1:]:
        assert pool_of(t) == side.cuda_stream
    assert pool_of(want[0]) != side.cuda_stream
    assert len(made) == (2 if what == "paged" else 0)


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.bfloat16])
def test_cache_offsets_behind_the_rows_are_reported(cuda_lib, dtype):
    """A sequence that ends behind the rows that are given is left out and reported, in
    append and in gather; the others are not touched by that."""
    g = gen(2)
    k, v = normal(g, 50, 2, 64), normal(g, 50, 2, 64)
    table, lens = ints([[0, 1], [2, 3], [4, 5]]), ints([20, 32, 10])
    cu, broken = ints([0, 20, 40, 50]), ints([0, 20, 60, 70])
    whole, cache = (cuda_lib.make_kv_cache(6, 16, 2, 64, dtype=dtype) for _ in range(2))
    cuda_lib.kv_cache_append(whole, k, v, lens, table, cu)
    cuda_lib.sync_status()
    before = [t.view(torch.uint8).clone() for t in cache.tensors() if t is not None]
    cuda_lib.kv_cache_append(cache, k, v, lens, table, broken)
    with pytest.raises(cuda_lib.WanvaeError) as ei:
        cuda_lib.sync_status()
    assert ei.value.status == cuda_lib.ERR_CUDA
    for a, b, c in zip((t for t in cache.tensors() if t is not None),
                       (t for t in whole.tensors() if t is not None), before):
        a, b = a.view(torch.uint8), b.view(torch.uint8)
        assert torch.equal(a[:2], b[:2]) and torch.equal(a[2:], c[2:])
    want_k, want_v = cuda_lib.kv_cache_gather(whole, table, cu, total=50)
    cuda_lib.sync_status()
    out_k, out_v = torch.full_like(want_k, 7.0), torch.full_like(want_v, 7.0)
    cuda_lib.kv_cache_gather(whole, table, broken, k=out_k, v=out_v)
    with pytest.raises(cuda_lib.WanvaeError):
        cuda_lib.sync_status()
    for got, want in ((out_k, want_k), (out_v, want_v)):
        assert torch.equal(got[:20], want[:20]) and torch.all(got[20:] == 7.0)


def test_paged_workspace_with_gaps_is_refused(cuda_lib):
    """Its bytes would not be where its elements are."""
    cache = cuda_lib.make_kv_cache(3, 16, 2, 64)
    q, table, lens = normal(gen(3), 1, 2, 64), ints([[0, 1, 2]]), ints([0])
    ws = cuda_lib.make_paged_attention_workspace(q, cache)
    cuda_lib.paged_attention(q, cache, lens, table, workspace=ws)
    cuda_lib.sync_status()
    with pytest.raises(cuda_lib.WanvaeError) as ei:
        cuda_lib.paged_attention(q, cache, lens, table,
                                 workspace=torch.cat([ws, ws])[::2])
    assert ei.value.status == cuda_lib.ERR_INVALID_ARG
