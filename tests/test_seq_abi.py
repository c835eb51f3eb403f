"""The sequence operators without a GPU: every refusal that the host can make,
before anything touches CUDA."""
import ctypes
import math

import pytest
import torch

from video_vae_causal_gb300 import build as libbuild
from video_vae_causal_gb300 import wanvae
from video_vae_causal_gb300.wanvae import (ERR_INVALID_ARG, ERR_MISALIGNED, ERR_UNSUPPORTED,
                                           ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return wanvae.load()


# 16-byte aligned fake device addresses, 256 MB apart (never dereferenced)
Q, K, V, O, W, L, P, C, KE, VE = (0x10000000 * (i + 1) for i in range(10))


def attention(lib, **edit):
    a = dict(q=Q, qs=256, k=K, ks=128, v=V, vs=128, out=O, os=256, cq=C, ck=C, n=2, tq=100,
             tk=100, hq=4, hk=2, d=64, scale=0.125, causal=1, stream=None)
    a.update(edit)
    return lib.wanvae_packed_attention(*a.values())


@pytest.mark.parametrize("edit,want", [
    (dict(q=None), ERR_INVALID_ARG), (dict(k=None), ERR_INVALID_ARG),
    (dict(v=None), ERR_INVALID_ARG), (dict(out=None), ERR_INVALID_ARG),
    (dict(cq=None), ERR_INVALID_ARG), (dict(ck=None), ERR_INVALID_ARG),
    (dict(n=0), ERR_INVALID_ARG), (dict(tq=0), ERR_INVALID_ARG), (dict(tk=-1), ERR_INVALID_ARG),
    (dict(tq=2 ** 31), ERR_INVALID_ARG), (dict(hq=3), ERR_INVALID_ARG),
    (dict(hk=0), ERR_INVALID_ARG), (dict(scale=0.0), ERR_INVALID_ARG),
    (dict(scale=math.nan), ERR_INVALID_ARG), (dict(scale=math.inf), ERR_INVALID_ARG),
    (dict(d=96), ERR_UNSUPPORTED), (dict(hq=258, qs=258 * 64, os=258 * 64), ERR_UNSUPPORTED),
    (dict(qs=248), ERR_INVALID_ARG), (dict(qs=260), ERR_INVALID_ARG),
    (dict(ks=120), ERR_INVALID_ARG), (dict(vs=132), ERR_INVALID_ARG),
    (dict(os=0), ERR_INVALID_ARG), (dict(q=Q + 8), ERR_MISALIGNED),
    (dict(cq=C + 2), ERR_MISALIGNED), (dict(out=Q + 512), ERR_INVALID_ARG),
    (dict(out=V + 1024), ERR_INVALID_ARG)])
def test_packed_attention_refuses(lib, edit, want):
    assert attention(lib, **edit) == want


def desc(**edit):
    d = dict(k=K, v=V, k_exp=KE, v_exp=VE, n_pages=4, page_size=16, n_kv_heads=2, head_dim=64,
             dt=wanvae.E4M3)
    d.update(edit)
    return ctypes.byref(wanvae.KvCacheDesc(*d.values()))


CACHES = [
    (dict(k=None), ERR_INVALID_ARG), (dict(v=None), ERR_INVALID_ARG),
    (dict(k_exp=None), ERR_INVALID_ARG), (dict(dt=wanvae.BF16), ERR_INVALID_ARG),
    (dict(dt=wanvae.F32), ERR_INVALID_ARG), (dict(dt=9), ERR_INVALID_ARG),
    (dict(n_pages=0), ERR_INVALID_ARG), (dict(n_kv_heads=0), ERR_INVALID_ARG),
    (dict(page_size=0), ERR_INVALID_ARG), (dict(page_size=8), ERR_UNSUPPORTED),
    (dict(page_size=48), ERR_UNSUPPORTED), (dict(page_size=2048), ERR_UNSUPPORTED),
    (dict(head_dim=32), ERR_UNSUPPORTED), (dict(v=K + 64), ERR_INVALID_ARG),
    (dict(k=K + 4), ERR_MISALIGNED), (dict(v_exp=VE + 1), ERR_MISALIGNED),
    (dict(v_exp=KE), ERR_INVALID_ARG)]


def append(lib, cache=None, **edit):
    a = dict(k=Q, ks=128, v=O, vs=128, lens=L, table=P, pages=2, cu=C, n=2, total=10, stream=None)
    a.update(edit)
    return lib.wanvae_kv_cache_append(cache or desc(), *a.values())


def gather(lib, cache=None, **edit):
    a = dict(table=P, pages=2, cu=C, n=2, total=10, k=Q, ks=128, v=O, vs=128, stream=None)
    a.update(edit)
    return lib.wanvae_kv_cache_gather(cache or desc(), *a.values())


def decode(lib, cache=None, **edit):
    n = lib.wanvae_paged_attention_workspace_size(4, 2, 64)
    a = dict(q=Q, qs=256, cache=cache or desc(), lens=L, table=P, pages=2, n=2, hq=4, scale=0.125,
             out=O, os=256, ws=W, bytes=n, stream=None)
    a.update(edit)
    return lib.wanvae_paged_attention(*a.values())


@pytest.mark.parametrize("edit,want", CACHES)
def test_bad_caches_are_refused(lib, edit, want):
    assert append(lib, desc(**edit)) == want
    assert gather(lib, desc(**edit)) == want
    assert decode(lib, desc(**edit)) == want


@pytest.mark.parametrize("edit,want", [
    (dict(k=None), ERR_INVALID_ARG), (dict(v=None), ERR_INVALID_ARG),
    (dict(table=None), ERR_INVALID_ARG), (dict(pages=0), ERR_INVALID_ARG),
    (dict(n=0), ERR_INVALID_ARG), (dict(total=0), ERR_INVALID_ARG),
    (dict(ks=120), ERR_INVALID_ARG), (dict(vs=129), ERR_INVALID_ARG),
    (dict(k=Q + 2), ERR_MISALIGNED), (dict(table=P + 1), ERR_MISALIGNED),
    (dict(v=V), ERR_INVALID_ARG)])
def test_append_and_gather_refuse(lib, edit, want):
    assert append(lib, **edit) == want
    assert gather(lib, **edit) == want


def test_no_cache_is_refused(lib):
    n = lib.wanvae_paged_attention_workspace_size(4, 2, 64)
    assert lib.wanvae_paged_attention(Q, 256, None, L, P, 2, 2, 4, 0.125, O, 256, W, n,
                                      None) == ERR_INVALID_ARG
    assert lib.wanvae_kv_cache_append(None, Q, 128, O, 128, L, P, 2, C, 2, 10,
                                      None) == ERR_INVALID_ARG
    assert lib.wanvae_kv_cache_gather(None, P, 2, C, 2, 10, Q, 128, O, 128,
                                      None) == ERR_INVALID_ARG


@pytest.mark.parametrize("edit", [
    dict(v=Q + 240), dict(v=Q + 16), dict(v=Q + 256, ks=248, vs=248),
    dict(v=Q + 256, ks=256, vs=264), dict(v=Q + 512 - 16, ks=256, vs=256),
    dict(v=Q - 512 + 16, ks=256, vs=256)])
def test_gather_refuses_rows_that_collide(lib, edit):
    """10 rows of 2 heads of 64 elements (256 bytes) each."""
    assert gather(lib, **edit) == ERR_INVALID_ARG


@pytest.mark.parametrize("edit,want", [
    # 64 sequences of 2^20 rows with 64 query heads: fits 32 bits; 2^29 rows and more do not
    (dict(n=64, pages=2 ** 16, qs=64 * 64, os=64 * 64, hq=64, bytes=10 ** 8, ws=None), ERR_WORKSPACE),
    (dict(n=1, pages=2 ** 25, ws=None), ERR_UNSUPPORTED),
    (dict(n=65535, pages=2 ** 16, ws=None), ERR_UNSUPPORTED)])
def test_paged_attention_counts_in_32_bits(lib, edit, want):
    assert decode(lib, **edit) == want


def test_append_without_offsets_is_one_row_a_sequence(lib):
    assert append(lib, cu=None) == ERR_INVALID_ARG
    assert append(lib, lens=None) == ERR_INVALID_ARG
    assert gather(lib, cu=None) == ERR_INVALID_ARG
    assert gather(lib, v=Q) == ERR_INVALID_ARG


@pytest.mark.parametrize("edit,want", [
    (dict(q=None), ERR_INVALID_ARG), (dict(out=None), ERR_INVALID_ARG),
    (dict(lens=None), ERR_INVALID_ARG), (dict(table=None), ERR_INVALID_ARG),
    (dict(n=0), ERR_INVALID_ARG),
    (dict(n=65536), ERR_INVALID_ARG), (dict(pages=0), ERR_INVALID_ARG),
    (dict(pages=2 ** 30), ERR_UNSUPPORTED), (dict(hq=3), ERR_INVALID_ARG),
    (dict(scale=-1.0), ERR_INVALID_ARG), (dict(qs=128), ERR_INVALID_ARG),
    (dict(os=257), ERR_INVALID_ARG), (dict(ws=None), ERR_WORKSPACE),
    (dict(bytes=1000), ERR_WORKSPACE), (dict(ws=W + 16), ERR_MISALIGNED),
    (dict(q=Q + 4), ERR_MISALIGNED), (dict(out=Q), ERR_INVALID_ARG),
    (dict(out=K), ERR_INVALID_ARG), (dict(ws=Q), ERR_INVALID_ARG)])
def test_paged_attention_refuses(lib, edit, want):
    assert decode(lib, **edit) == want


def test_paged_attention_workspace_size(lib):
    size = wanvae.paged_attention_workspace_size
    assert size(32, 8, 128) > 0 and size(32, 8, 128) % 256 == 0
    assert size(16, 1, 128) > size(8, 1, 128) > size(8, 1, 64) > 0
    assert size(3, 2, 64) == size(4, 2, 96) == size(0, 1, 64) == size(4, 0, 64) == 0


def norm(lib, **edit):
    a = dict(x=Q, f=K, gp=C, gate=P, per=1, gn=L, y=V, n=O, dt=wanvae.BF16, tokens=100, ch=64,
             scale=1.0, eps=1e-12, stream=None)
    a.update(edit)
    return lib.wanvae_gated_residual_norm(*a.values())


@pytest.mark.parametrize("edit,want", [
    (dict(x=None), ERR_INVALID_ARG), (dict(f=None), ERR_INVALID_ARG),
    (dict(y=None), ERR_INVALID_ARG), (dict(n=None), ERR_INVALID_ARG),
    (dict(gn=None), ERR_INVALID_ARG), (dict(dt=wanvae.E4M3), ERR_INVALID_ARG),
    (dict(tokens=0), ERR_INVALID_ARG), (dict(tokens=2 ** 31), ERR_INVALID_ARG),
    (dict(ch=24), ERR_INVALID_ARG), (dict(ch=4112), ERR_INVALID_ARG),
    (dict(per=0), ERR_INVALID_ARG), (dict(eps=-1.0), ERR_INVALID_ARG),
    (dict(eps=math.nan), ERR_INVALID_ARG), (dict(scale=math.inf), ERR_INVALID_ARG),
    (dict(scale=math.nan), ERR_INVALID_ARG), (dict(gp=C + 4), ERR_MISALIGNED),
    (dict(y=V + 8), ERR_MISALIGNED), (dict(y=Q), ERR_INVALID_ARG), (dict(n=K), ERR_INVALID_ARG),
    (dict(n=V + 128), ERR_INVALID_ARG), (dict(gp=V + 64), ERR_INVALID_ARG),
    (dict(gp=V - 64), ERR_INVALID_ARG), (dict(gate=O - 99 * 256), ERR_INVALID_ARG),
    (dict(gate=O - 256, per=2 ** 62, gn=O), ERR_INVALID_ARG)])
def test_gated_norm_refuses(lib, edit, want):
    assert norm(lib, **edit) == want


def test_tensors_off_the_device_are_refused(lib):
    """The binding hands no host pointer to a kernel."""
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    cache = wanvae.make_kv_cache(2, 16, 2, 64, device="cpu")
    table = torch.zeros((1, 2), dtype=torch.int32)
    for call in (lambda: wanvae.packed_attention(q, q, q, cu),
                 lambda: wanvae.kv_cache_append(cache, q, q, cu[1:], table, cu),
                 lambda: wanvae.kv_cache_gather(cache, table, cu, total=4),
                 lambda: wanvae.paged_attention(q[:1], cache, cu[1:], table),
                 lambda: wanvae.gated_residual_norm(x, x)):
        with pytest.raises(wanvae.WanvaeError) as ei:
            call()
        assert ei.value.status == ERR_INVALID_ARG


def test_cache_tensors_have_to_fit():
    k = torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16)
    q8 = k.to(torch.float8_e4m3fn)
    e = torch.zeros((2, 2, 16), dtype=torch.uint8)
    wanvae.KVCache(k, k.clone())
    wanvae.KVCache(q8, q8.clone(), e, e.clone())
    for bad in ((k, k[:1]), (k, q8), (k.float(), k.float()), (q8, q8.clone()), (k, k.clone(), e, e),
                (q8, q8.clone(), e, e[:1]), (q8, q8.clone(), e.int(), e.int()),
                (k.transpose(1, 2), k.transpose(1, 2)), (k[0], k[1])):
        with pytest.raises(wanvae.WanvaeError):
            wanvae.KVCache(*bad)
