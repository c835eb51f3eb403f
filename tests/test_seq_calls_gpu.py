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
