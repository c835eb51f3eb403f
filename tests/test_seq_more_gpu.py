"""Cases of the sequence operators that lie between the ones of test_seq_gpu.py: rows that are
not finite.  References and bounds as there."""
import math

import pytest
import torch

from test_seq_gpu import DEV, DTYPES, attend, close, fill, gen, ints, normal, rows_of, widened

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


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
