"""What the norm and rotation of queries and keys, the pages of a cache and a cache in 4 bits
refuse on the host, before anything touches CUDA."""
import ctypes
import math

import pytest
import torch

from test_seq_abi import (C, K, KE, L, O, P, Q, V, VE, W, append, decode, desc, gather,
                          lib)  # noqa: F401 (lib: the fixture)
from video_vae_causal_gb300 import wanvae
from video_vae_causal_gb300.wanvae import (ERR_INVALID_ARG, ERR_MISALIGNED, ERR_UNSUPPORTED,
                                           ERR_WORKSPACE)

KO, VO, S, N, FR, NF = (0x10000000 * (i + 20) for i in range(6))


# ------------------------------------------------------------------ norm and rotation
def rotary(pairs=(32,), inv_freq=None, **edit):
    freq = [1.0] * 64 if inv_freq is None else inv_freq
    d = dict(inv_freq=(ctypes.c_double * 64)(*freq), axes=len(pairs),
             pairs=(ctypes.c_int64 * 4)(*pairs), interleaved=0)
    d.update(edit)
    return ctypes.byref(wanvae.RotaryDesc(*d.values()))


def rotate(lib, rot=None, **edit):
    a = dict(q=Q, qs=256, k=K, ks=128, gq=C, gk=L, rot=rot or rotary(), pos=P, qo=O, qos=256,
             ko=V, kos=128, dt=wanvae.BF16, tokens=100, hq=4, hk=2, d=64, eps=1e-12, stream=None)
    a.update(edit)
    return lib.wanvae_qk_norm_rotate(*a.values())


@pytest.mark.parametrize("edit,want", [
    (dict(q=None), ERR_INVALID_ARG), (dict(k=None), ERR_INVALID_ARG),
    (dict(qo=None), ERR_INVALID_ARG), (dict(ko=None), ERR_INVALID_ARG),
    (dict(pos=None), ERR_INVALID_ARG), (dict(hk=0), ERR_INVALID_ARG),
    (dict(k=None, ko=None, hk=0), ERR_INVALID_ARG),  # (a gamma for no keys)
    (dict(dt=wanvae.E4M3), ERR_INVALID_ARG), (dict(dt=9), ERR_INVALID_ARG),
    (dict(tokens=0), ERR_INVALID_ARG), (dict(tokens=2 ** 31), ERR_INVALID_ARG),
    (dict(hq=0), ERR_INVALID_ARG), (dict(hk=-1), ERR_INVALID_ARG),
    (dict(eps=-1.0), ERR_INVALID_ARG), (dict(eps=math.nan), ERR_INVALID_ARG),
    (dict(d=96), ERR_UNSUPPORTED), (dict(hq=65536, qs=65536 * 64, qos=65536 * 64), ERR_UNSUPPORTED),
    (dict(qs=248), ERR_INVALID_ARG), (dict(ks=120), ERR_INVALID_ARG), (dict(qos=260), ERR_INVALID_ARG),
    (dict(kos=0), ERR_INVALID_ARG), (dict(q=Q + 8), ERR_MISALIGNED), (dict(ko=V + 2), ERR_MISALIGNED),
    (dict(gq=C + 4), ERR_MISALIGNED), (dict(pos=P + 2), ERR_MISALIGNED),
    (dict(qo=Q + 512), ERR_INVALID_ARG), (dict(qo=Q, qos=264), ERR_INVALID_ARG),
    (dict(qo=K), ERR_INVALID_ARG), (dict(ko=Q), ERR_INVALID_ARG), (dict(ko=O + 256), ERR_INVALID_ARG),
    (dict(qo=Q + 256, qs=512, qos=504), ERR_INVALID_ARG),
    (dict(ko=Q + 496, qs=512, kos=512), ERR_INVALID_ARG),
    (dict(qo=C), ERR_INVALID_ARG), (dict(ko=L - 256), ERR_INVALID_ARG),
    (dict(qo=P), ERR_INVALID_ARG), (dict(ko=P + 256), ERR_INVALID_ARG)])
def test_rotation_refuses(lib, edit, want):  # noqa: F811
    assert rotate(lib, **edit) == want


@pytest.mark.parametrize("make,want", [
    (dict(pairs=(36,)), ERR_INVALID_ARG), (dict(pairs=(30,)), ERR_UNSUPPORTED),
    (dict(pairs=(20, 16)), ERR_INVALID_ARG), (dict(pairs=(-4, 8)), ERR_INVALID_ARG),
    (dict(pairs=(2 ** 62, 2 ** 62)), ERR_INVALID_ARG),
    (dict(axes=0), ERR_INVALID_ARG), (dict(axes=5), ERR_INVALID_ARG),
    (dict(inv_freq=[math.nan] * 64), ERR_INVALID_ARG),
    (dict(inv_freq=[1.0] * 31 + [math.inf] * 33), ERR_INVALID_ARG),
    (dict(inv_freq=[2.0 ** 20 + 1] * 64), ERR_INVALID_ARG)])
def test_rotation_refuses_frequencies(lib, make, want):  # noqa: F811
    inv = make.pop("inv_freq", None)
    rot = rotary(make.pop("pairs", (32,)), inv, **make)
    assert rotate(lib, rot) == want


def test_rotation_without_frequencies(lib):  # noqa: F811
    assert rotate(lib, rotary(inv_freq=None, **{}), q=None) == ERR_INVALID_ARG
    none = ctypes.byref(wanvae.RotaryDesc(None, 1, (ctypes.c_int64 * 4)(32), 0))
    assert rotate(lib, none) == ERR_INVALID_ARG
    assert lib.wanvae_qk_norm_rotate(Q, 256, K, 128, C, L, None, P, O, 256, V, 128, 0, 100, 4, 2, 64,
                                     1e-12, None) == ERR_INVALID_ARG


def test_rotary_checks_its_arguments():
    r = wanvae.Rotary([12, 10, 10], theta=100.0)
    assert r.pairs == [12, 10, 10] and len(r.inv_freq) == 32
    assert r.inv_freq[0] == r.inv_freq[12] == r.inv_freq[22] == 1.0
    assert r.inv_freq[13] == 100.0 ** (-1 / 10)
    assert wanvae.Rotary(32).pairs == [32]
    for bad in (dict(pairs=[]), dict(pairs=[1] * 5), dict(pairs=[-4]), dict(pairs=4, inv_freq=[1.0])):
        with pytest.raises(wanvae.WanvaeError):
            wanvae.Rotary(**bad)


# ------------------------------------------------------------------ pages
def pool(**edit):
    d = dict(free=FR, n_free=NF, n_pages=50, page=16)
    d.update(edit)
    return ctypes.byref(wanvae.KvPagePoolDesc(*d.values()))


def extend(lib, p=None, **edit):
    a = dict(lens=L, new=N, table=P, pages=8, n=4, total=20, lo=L, no=NF, cu=C, taken=W, pos=Q, slots=S,
             stream=None)
    a.update(edit)
    return lib.wanvae_kv_pages_extend(p or pool(), *a.values())


def release(lib, p=None, **edit):
    a = dict(lens=L, done=N, table=P, pages=8, n=4, lo=L, no=NF, stream=None)
    a.update(edit)
    return lib.wanvae_kv_pages_release(p or pool(), *a.values())


@pytest.mark.parametrize("make,want", [
    (dict(free=None), ERR_INVALID_ARG), (dict(n_free=None), ERR_INVALID_ARG),
    (dict(n_pages=0), ERR_INVALID_ARG), (dict(n_pages=2 ** 31), ERR_INVALID_ARG),
    (dict(page=0), ERR_INVALID_ARG), (dict(page=24), ERR_UNSUPPORTED), (dict(page=8), ERR_UNSUPPORTED),
    (dict(page=2048), ERR_UNSUPPORTED), (dict(free=FR + 2), ERR_MISALIGNED),
    (dict(n_free=NF + 1), ERR_MISALIGNED), (dict(free=L), ERR_INVALID_ARG),
    (dict(n_free=P + 4), ERR_INVALID_ARG), (dict(free=P - 4), ERR_INVALID_ARG)])
def test_bad_pools_are_refused(lib, make, want):  # noqa: F811
    edit = {} if "n_free" not in make else dict(no=make["n_free"] or NF)
    if make != dict(n_free=P + 4):  # (release reads the table)
        assert release(lib, pool(**make), **edit) == want
    assert extend(lib, pool(**make), **edit) == want


@pytest.mark.parametrize("edit,want", [
    (dict(lens=None), ERR_INVALID_ARG), (dict(table=None), ERR_INVALID_ARG),
    (dict(lo=None), ERR_INVALID_ARG), (dict(no=None), ERR_INVALID_ARG),
    (dict(pages=0), ERR_INVALID_ARG), (dict(n=0), ERR_INVALID_ARG), (dict(n=16385), ERR_UNSUPPORTED),
    (dict(pages=2 ** 27), ERR_UNSUPPORTED), (dict(lens=L + 1), ERR_MISALIGNED),
    (dict(table=P + 2), ERR_MISALIGNED), (dict(lo=L + 4), ERR_INVALID_ARG),
    (dict(lo=L - 12), ERR_INVALID_ARG), (dict(no=L), ERR_INVALID_ARG), (dict(lo=NF), ERR_INVALID_ARG),
    (dict(lo=P + 124), ERR_INVALID_ARG), (dict(no=FR + 196), ERR_INVALID_ARG)])
def test_pages_refuse(lib, edit, want):  # noqa: F811
    assert extend(lib, **edit) == want
    assert release(lib, **edit) == want


@pytest.mark.parametrize("edit,want", [
    (dict(new=None), ERR_INVALID_ARG), (dict(cu=None), ERR_INVALID_ARG),
    (dict(taken=None), ERR_INVALID_ARG), (dict(pos=None), ERR_INVALID_ARG),
    (dict(slots=None), ERR_INVALID_ARG), (dict(total=0), ERR_INVALID_ARG),
    (dict(total=2 ** 31), ERR_INVALID_ARG), (dict(slots=S + 4), ERR_MISALIGNED),
    (dict(pos=Q + 1), ERR_MISALIGNED), (dict(cu=L), ERR_INVALID_ARG), (dict(cu=L - 16), ERR_INVALID_ARG),
    (dict(taken=N + 12), ERR_INVALID_ARG), (dict(pos=C + 16), ERR_INVALID_ARG),
    (dict(slots=Q + 72), ERR_INVALID_ARG), (dict(slots=FR), ERR_INVALID_ARG),
    (dict(taken=NF), ERR_INVALID_ARG), (dict(pos=P + 64), ERR_INVALID_ARG)])
def test_extend_refuses(lib, edit, want):  # noqa: F811
    assert extend(lib, **edit) == want


def test_release_refuses(lib):  # noqa: F811
    assert release(lib, done=None) == ERR_INVALID_ARG
    assert release(lib, done=L + 3) == ERR_INVALID_ARG
    assert release(lib, done=FR) == ERR_INVALID_ARG
    assert lib.wanvae_kv_pages_release(None, L, N, P, 8, 4, L, NF, None) == ERR_INVALID_ARG
    assert lib.wanvae_kv_pages_extend(None, L, N, P, 8, 4, 20, L, NF, C, W, Q, S,
                                      None) == ERR_INVALID_ARG


# ------------------------------------------------------------------ a cache in 4 bits
def desc4(**edit):
    d = dict(dt=wanvae.E2M1, k_off=KO, v_off=VO)
    d.update(edit)
    return desc(**d)


CACHES = [
    (dict(k_off=None), ERR_INVALID_ARG), (dict(v_off=None), ERR_INVALID_ARG),
    (dict(k_exp=None), ERR_INVALID_ARG), (dict(k=None), ERR_INVALID_ARG),
    (dict(k_off=KO + 8), ERR_MISALIGNED), (dict(v_off=VO + 1), ERR_MISALIGNED),
    (dict(v_off=KO), ERR_INVALID_ARG), (dict(k_off=K), ERR_INVALID_ARG),
    (dict(v_off=VE + 64), ERR_INVALID_ARG), (dict(v_exp=KE), ERR_INVALID_ARG),
    (dict(v=K + 4080), ERR_INVALID_ARG),  # (4 pages of 2 heads of 16 rows of 32 bytes)
    (dict(head_dim=32), ERR_UNSUPPORTED), (dict(page_size=8), ERR_UNSUPPORTED)]


def write(lib, cache=None, **edit):
    a = dict(k=Q, ks=128, v=O, vs=128, slots=S, total=10, stream=None)
    a.update(edit)
    return lib.wanvae_kv_cache_write(cache or desc4(), *a.values())


@pytest.mark.parametrize("edit,want", CACHES)
def test_bad_caches_are_refused(lib, edit, want):  # noqa: F811
    for call in (append, gather, decode, write):
        assert call(lib, desc4(**edit)) == want


def test_what_lies_over_the_offsets_is_refused(lib):  # noqa: F811
    assert append(lib, desc4(), lens=KO) == ERR_INVALID_ARG
    assert gather(lib, desc4(), k=VO) == ERR_INVALID_ARG
    assert decode(lib, desc4(), out=VO) == ERR_INVALID_ARG
    assert decode(lib, desc4(), ws=KO) == ERR_INVALID_ARG
    assert decode(lib, desc4(), ws=None) == ERR_WORKSPACE
    # the other types have no offsets, and do not look at them
    assert gather(lib, desc(k_off=K, v_off=3), n=0) == ERR_INVALID_ARG
    assert decode(lib, desc(k_off=K, v_off=3), ws=None) == ERR_WORKSPACE


@pytest.mark.parametrize("cache", [desc4, desc])
@pytest.mark.parametrize("edit,want", [
    (dict(k=None), ERR_INVALID_ARG), (dict(v=None), ERR_INVALID_ARG), (dict(slots=None), ERR_INVALID_ARG),
    (dict(total=0), ERR_INVALID_ARG), (dict(total=2 ** 31), ERR_INVALID_ARG),
    (dict(ks=120), ERR_INVALID_ARG), (dict(vs=130), ERR_INVALID_ARG), (dict(k=Q + 8), ERR_MISALIGNED),
    (dict(slots=S + 4), ERR_MISALIGNED), (dict(k=V), ERR_INVALID_ARG), (dict(slots=KE), ERR_INVALID_ARG),
    (dict(v=KE - 128), ERR_INVALID_ARG)])
def test_write_refuses(lib, cache, edit, want):  # noqa: F811
    assert write(lib, cache(), **edit) == want


def test_cache_tensors_have_to_fit():
    shape = (2, 3, 16)
    k = torch.zeros((*shape, 32), dtype=torch.uint8)
    e, o = torch.zeros(shape, dtype=torch.uint8), torch.zeros((*shape, 2), dtype=torch.uint8)
    c = wanvae.KVCache(k, k.clone(), e, e.clone(), o, o.clone())
    assert c.head_dim == 64 and c.heads == 3 and c.page_size == 16
    made = wanvae.make_kv_cache(2, 16, 3, 128, dtype=torch.uint8, device="cpu")
    assert made.k.shape == (*shape, 64) and made.v_off.shape == (*shape, 4) and made.head_dim == 128
    bf, q8 = torch.zeros((*shape, 64), dtype=torch.bfloat16), torch.zeros((*shape, 64))
    q8 = q8.to(torch.float8_e4m3fn)
    for bad in ((k, k), (k, k, e, e), (k, k, None, None, o, o), (k, k, e, e, o, o[..., :1]),
                (k, k, e, e, o.int(), o.int()), (k, k, e, e, o, o.transpose(0, 1)),
                (bf, bf, None, None, o, o), (q8, q8, e, e, o, o), (k, k, e, e, o, None)):
        with pytest.raises(wanvae.WanvaeError):
            wanvae.KVCache(*bad)


def test_pool_tensors_have_to_fit():
    p = wanvae.make_kv_page_pool(5, 16, device="cpu")
    assert p.free.tolist() == [4, 3, 2, 1, 0] and p.n_free.tolist() == [5]
    for free, n in ((p.free.long(), p.n_free), (p.free, p.n_free.long()), (p.free, p.free),
                    (p.free[::2], p.n_free), (p.free.view(1, 5), p.n_free)):
        with pytest.raises(wanvae.WanvaeError):
            wanvae.KVPagePool(free, n, 16)


def test_tensors_off_the_device_are_refused(lib):  # noqa: F811
    """The binding hands no host pointer to a kernel."""
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    cache = wanvae.make_kv_cache(2, 16, 2, 64, dtype=torch.uint8, device="cpu")
    p = wanvae.make_kv_page_pool(2, 16, device="cpu")
    table = torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: wanvae.qk_norm_rotate(q, q, i, wanvae.Rotary(32)),
                 lambda: wanvae.kv_cache_write(cache, q, q, i.long()),
                 lambda: wanvae.kv_pages_extend(p, i, i, table, total=4),
                 lambda: wanvae.kv_pages_release(p, i, i.to(torch.uint8), table)):
        with pytest.raises(wanvae.WanvaeError) as ei:
            call()
        assert ei.value.status == ERR_INVALID_ARG


@pytest.mark.parametrize("dtype,code", [(torch.uint8, 127 - 94), (torch.float8_e4m3fn, 127)])
def test_an_empty_caches_rows_have_the_scale_of_zeros(dtype, code):
    cache = wanvae.make_kv_cache(2, 16, 3, 64, dtype=dtype, device="cpu")
    for e in (cache.k_exp, cache.v_exp):
        assert (e.view(torch.uint8) == code).all()
    assert all((t.view(torch.uint8) == 0).all() for t in cache.tensors()
               if t is not cache.k_exp and t is not cache.v_exp)
