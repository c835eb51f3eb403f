"""The norm of query and key heads with their rotation on the GPU, against the definition
in 64 bits.

Tolerance.  Before the one rounding of the output (u = 2^-8 in bf16, 2^-24 in fp32, relative)
a normed element n is off by less than 2^-20 of itself: the sum of D <= 128 squares goes
through 4 + 5 roundings of 2^-24, of which the root leaves half, the reciprocal root is off by
two units (2^-22), and six more roundings follow (weight times sqrt(D), times a cosine, the
product, the sum, times the root).  A sine or cosine is off by less than 2^-22 in fp32: the angle
by 2^-33 of a turn and the 2^-25 of half a turn that an fp32 angle rounds to (pi 2^-25), the
function itself by two units of 2^-24; and by less than 2^-20 for bf16 rows: the angle's product
with pi rounds (pi 2^-23 with pi's own rounding), and the fast functions are off by 2^-21.19 at
most.  With y = n_a cos - n_b sin the error stays below u |y| + (2^-20 + trig) (|n_a| + |n_b|).
"""
import math
from fractions import Fraction

import pytest
import torch

from test_seq_gpu import DEV, gen, normal

pytestmark = pytest.mark.gpu

TURN = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
REST = {torch.float32: 2.0 ** -20 + 2.0 ** -22, torch.bfloat16: 2.0 ** -20 + 2.0 ** -20}


def angles(positions, rotary):
    """The pairs' angles [T, P] in 64 bits, reduced exactly."""
    axis = [a for a, n in enumerate(rotary.pairs) for _ in range(n)]
    rows = positions.view(positions.shape[0], -1).tolist()
    return torch.tensor([[float(Fraction(rotary.inv_freq[p]) * row[a] % TURN)
                          for p, a in enumerate(axis)] for row in rows],
                        dtype=torch.float64, device=DEV).view(len(rows), len(axis))


def definition(x, gamma, angle, interleaved, eps=1e-12):
    """(y, |n_a| + |n_b|) in 64 bits."""
    n = x.double()
    if gamma is not None:
        norm = n.square().sum(-1, keepdim=True).sqrt().clamp_min(eps)
        n = n / norm * math.sqrt(x.shape[-1]) * gamma.double()
    P = angle.shape[1]
    a = list(range(0, 2 * P, 2)) if interleaved else list(range(P))
    b = list(range(1, 2 * P, 2)) if interleaved else list(range(P, 2 * P))
    y, size = n.clone(), n.abs()
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    y[..., a], y[..., b] = n[..., a] * c - n[..., b] * s, n[..., b] * c + n[..., a] * s
    both = n[..., a].abs() + n[..., b].abs()
    size[..., a], size[..., b] = both, both
    return y, size


def check(got, want, size, what=""):
    u = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    over = (got.double() - want).abs() - (u * want.abs() + REST[got.dtype] * size)
    assert torch.isfinite(got).all(), what
    assert (over <= 0).all(), f"{what}: over by {over.max().item():.3e}"


def run(lib, T, hq, hk, D, rotary, dtype=torch.bfloat16, positions=None, seed=0, gammas=True, **kw):
    g = gen(seed)
    qkv = normal(g, T, hq + 2 * hk + 1, D, dtype=dtype)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    if positions is None:
        shape = (T, len(rotary.pairs))
        positions = torch.randint(0, 8192, shape, generator=g, device=DEV, dtype=torch.int32)
    gq, gk = (torch.rand(D, generator=g, device=DEV) + 0.5 for _ in range(2))
    if not gammas:
        gq = gk = None
    angle = angles(positions, rotary)
    want = [definition(x, gm, angle, rotary.interleaved) for x, gm in ((q, gq), (k, gk))]
    rest = qkv[:, hq + hk:].clone()
    qo, ko = lib.qk_norm_rotate(q, k if hk else None, positions, rotary, gq, gk if hk else None, **kw)
    lib.sync_status()
    check(qo, *want[0], "q")
    if hk:
        check(ko, *want[1], "k")
    else:
        assert ko is None
    assert torch.equal(qkv[:, hq + hk:], rest)
    return q, k, qo, ko


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,pairs", [(64, [32]), (128, [64]), (128, [32]), (64, [4]), (128, [4]),
                                     (64, [12, 10, 10]), (128, [22, 21, 21]), (128, [0, 8, 0, 4]),
                                     (64, [0])])
def test_rotations(cuda_lib, D, pairs, interleaved, dtype):
    run(cuda_lib, 37, 5, 2, D, cuda_lib.Rotary(pairs, interleaved=interleaved), dtype, seed=D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,hq,hk", [(1, 1, 0), (1, 1, 1), (2, 3, 1), (64, 32, 8), (3, 130, 7),
                                     (2600, 12, 12), (6000, 1, 1)])
def test_sizes(cuda_lib, D, T, hq, hk):
    run(cuda_lib, T, hq, hk, D, cuda_lib.Rotary(D // 2), seed=T + hq)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_far_positions(cuda_lib, dtype):
    """Angles hold to the last position of 32 bits, negative ones too."""
    at = [0, 1, -1, 131040, -131040, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345]
    pos = torch.tensor(at, dtype=torch.int32, device=DEV)
    run(cuda_lib, len(at), 3, 2, 128, cuda_lib.Rotary(64), dtype, positions=pos)


def test_given_frequencies(cuda_lib):
    freq = [0.0, 1.0, -2.5, math.pi, 1e-7, 1234.5678, 2.0 ** 20, 1e-30]
    pos = torch.tensor([0, 3, 99999, -7, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    run(cuda_lib, 5, 2, 1, 64, cuda_lib.Rotary([8], inv_freq=freq), torch.float32, positions=pos)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rotation_without_norm(cuda_lib, interleaved, dtype):
    run(cuda_lib, 65, 4, 2, 128, cuda_lib.Rotary([40], interleaved=interleaved), dtype, gammas=False)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_in_place_and_between_other_rows(cuda_lib, D, interleaved):
    g, T, hq, hk = gen(5), 300, 6, 2
    rotary = cuda_lib.Rotary(D // 2, interleaved=interleaved)
    qkv = normal(g, T, hq + 2 * hk, D)
    pos = torch.randint(0, 999, (T,), generator=g, device=DEV, dtype=torch.int32)
    gamma = torch.rand(D, generator=g, device=DEV) + 0.5
    want = cuda_lib.qk_norm_rotate(qkv[:, :hq], qkv[:, hq:hq + hk], pos, rotary, gamma, gamma)
    v = qkv[:, hq + hk:].clone()
    other = torch.full((T, hq + hk, D), 7.0, dtype=torch.bfloat16, device=DEV)
    cuda_lib.qk_norm_rotate(qkv[:, :hq], qkv[:, hq:hq + hk], pos, rotary, gamma, gamma,
                            q_out=other[:, hk:], k_out=other[:, :hk])
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    got = cuda_lib.qk_norm_rotate(q, k, pos, rotary, gamma, gamma, q_out=q, k_out=k)
    cuda_lib.sync_status()
    assert got[0] is q and got[1] is k
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(other[:, hk:], want[0]) and torch.equal(other[:, :hk], want[1])
    assert torch.equal(qkv[:, hq + hk:], v)


def test_zeros_small_heads_and_values_that_are_not_finite(cuda_lib):
    """A head of zeros stays zeros; one of norm below eps is divided by eps; NaN and
    infinities stay in their head; without a norm in their pair."""
    D, rotary = 64, cuda_lib.Rotary(16)
    x = normal(gen(1), 4, 3, D, dtype=torch.float32)
    x[0, 0] = 0
    x[1, 0] = 1e-20
    x[2, 0, 5] = math.nan
    x[3, 0, 40] = math.inf
    pos = torch.tensor([3, 4, 5, 6], dtype=torch.int32, device=DEV)
    gamma = torch.ones(D, device=DEV)
    y, _ = cuda_lib.qk_norm_rotate(x, None, pos, rotary, gamma, eps=1e-6)
    cuda_lib.sync_status()
    assert (y[0, 0] == 0).all()
    want, size = definition(x[1:2], gamma, angles(pos[1:2], rotary), False, eps=1e-6)
    check(y[1:2], want, size)
    assert y[2, 0].isnan().all() and y[3, 0, 40].isnan()
    assert torch.isfinite(y[:, 1:]).all()
    z, _ = cuda_lib.qk_norm_rotate(x, None, pos, rotary)
    bad = torch.zeros((4, 3, D), dtype=torch.bool, device=DEV)
    bad[2, 0, [5, 21]] = True    # a pair that turns
    bad[3, 0, 40] = True         # an element that does not
    assert torch.equal(~torch.isfinite(z), bad) and z[3, 0, 40] == math.inf


def test_another_stream_and_a_captured_graph(cuda_lib):
    g, T, D = gen(9), 50, 128
    rotary = cuda_lib.Rotary(64)
    q, k = normal(g, T, 8, D), normal(g, T, 2, D)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    gamma = torch.ones(D, device=DEV)
    want = cuda_lib.qk_norm_rotate(q, k, pos, rotary, gamma, gamma)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = cuda_lib.qk_norm_rotate(q, k, pos, rotary, gamma, gamma, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(q), torch.empty_like(k)
    with torch.cuda.graph(graph):
        cuda_lib.qk_norm_rotate(q, k, pos, rotary, gamma, gamma, q_out=out[0], k_out=out[1])
    del rotary  # (its frequencies are in the graph)
    pos += 1000
    graph.replay()
    again = cuda_lib.qk_norm_rotate(q, k, pos, cuda_lib.Rotary(64), gamma, gamma)
    cuda_lib.sync_status()
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])
    assert not torch.equal(out[0], want[0])


def test_offsets_beyond_32_bits(cuda_lib):
    """A row's bytes from the first pass 2^32."""
    T, D, stride = 3, 64, 2 ** 30 + 2 ** 29
    buf = torch.zeros(2 * stride + 4 * D, dtype=torch.bfloat16, device=DEV)
    q = buf.as_strided((T, 2, D), (stride, D, 1))
    x = normal(gen(2), T, 2, D)
    q.copy_(x)
    pos = torch.tensor([5, 6, 7], dtype=torch.int32, device=DEV)
    rotary, gamma = cuda_lib.Rotary(32), torch.ones(D, device=DEV)
    got, _ = cuda_lib.qk_norm_rotate(q, None, pos, rotary, gamma)
    cuda_lib.qk_norm_rotate(q, None, pos, rotary, gamma, q_out=q)
    cuda_lib.sync_status()
    want, size = definition(x, gamma, angles(pos, rotary), False)
    check(got, want, size)
    assert torch.equal(q, got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_negative_frequencies_turn_back(cuda_lib, dtype):
    """-f at a position is f at the negated one, bit for bit, however far it lies."""
    freq = [0.3, 1e-3, 1e-7, 2.5, 1.0, 0.7311, 1e-12, 1234.5678]
    pos = torch.tensor([1, 12345, 99999, 2 ** 31 - 1, 2 ** 31 - 1000, 1 - 2 ** 31, -7],
                       dtype=torch.int32, device=DEV)
    x = normal(gen(6), len(pos), 2, 64, dtype=dtype)
    back, _ = cuda_lib.qk_norm_rotate(x, None, pos, cuda_lib.Rotary([8], inv_freq=[-f for f in freq]))
    want, _ = cuda_lib.qk_norm_rotate(x, None, -pos, cuda_lib.Rotary([8], inv_freq=freq))
    cuda_lib.sync_status()
    assert torch.equal(back, want)
    angle = angles(pos, cuda_lib.Rotary([8], inv_freq=[-f for f in freq]))
    check(back, *definition(x, None, angle, False))
