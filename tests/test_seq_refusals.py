"""More of what the sequence operators refuse on the host, before anything touches CUDA
(the calls and fake addresses of test_seq_abi.py)."""
import pytest
import torch

from test_seq_abi import (C, K, KE, L, O, P, Q, V, VE, W, append, attention, decode, gather,
                          lib)  # noqa: F401 (lib: the fixture)
from video_vae_causal_gb300 import wanvae
from video_vae_causal_gb300.wanvae import ERR_INVALID_ARG


@pytest.mark.parametrize("edit", [
    dict(cq=O), dict(ck=O + 256), dict(cq=O - 8), dict(ck=O + 99 * 512 + 508)])
def test_packed_attention_refuses_offsets_in_its_output(lib, edit):  # noqa: F811
    """Written while they are read: 100 tokens of 4 heads of 64, 3 offsets."""
    assert attention(lib, **edit) == ERR_INVALID_ARG


@pytest.mark.parametrize("edit", [
    dict(lens=K), dict(table=V + 4096), dict(cu=KE), dict(lens=VE + 16), dict(table=K - 12),
    dict(cu=V - 8)])
def test_append_refuses_lengths_offsets_and_pages_in_the_cache(lib, edit):  # noqa: F811
    assert append(lib, **edit) == ERR_INVALID_ARG


@pytest.mark.parametrize("edit", [
    dict(cu=Q), dict(table=Q + 128), dict(cu=O + 9 * 256), dict(table=O - 12), dict(cu=O - 8)])
def test_gather_refuses_offsets_and_pages_in_its_outputs(lib, edit):  # noqa: F811
    """10 rows of 256 bytes, 3 offsets, 2 x 2 pages."""
    assert gather(lib, **edit) == ERR_INVALID_ARG


@pytest.mark.parametrize("edit", [
    dict(lens=O), dict(table=O + 512), dict(lens=W), dict(table=W + 1024), dict(table=W - 12),
    dict(lens=O - 4)])
def test_paged_attention_refuses_lengths_and_pages_in_what_it_writes(lib, edit):  # noqa: F811
    """2 sequences: lengths of 8 bytes, 2 x 2 pages."""
    assert decode(lib, **edit) == ERR_INVALID_ARG


@pytest.mark.parametrize("stride", [0, 4, 132, 1000])
def test_one_token_s_stride_means_nothing(stride):
    """A single token out of a buffer whose rows would not do for several."""
    buf = torch.zeros(4096, dtype=torch.bfloat16)
    assert wanvae._heads("", buf.as_strided((1, 2, 64), (stride, 64, 1))) == 128
    assert wanvae._heads("", buf.as_strided((2, 2, 64), (132, 64, 1))) == 132


def test_a_stream_of_another_device_is_refused():
    """The launch would fail there, and leave its error for the next one to find."""
    class Stream:
        cuda_stream, device_index = 7, 1
    assert wanvae._raw_stream("", Stream, 1) == 7
    with pytest.raises(wanvae.WanvaeError) as ei:
        wanvae._raw_stream("", Stream, 0)
    assert ei.value.status == ERR_INVALID_ARG
