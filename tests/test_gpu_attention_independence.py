"""A row of cache_attention does not depend on the other sequences' queries, also
where a prefix shared by all is computed for several sequences' rows at once: its
result stays the same to the bit.  On the GPU."""
import numpy as np
import pytest
import torch

from bit_gemm_block_amd import decode as D
from test_gpu_attention import bar, check, dev, host, make_cache, queries, tables_of

pytestmark = pytest.mark.gpu


# Rows of a cache head: 16 in one tile, which waves share, and more.
@pytest.mark.parametrize("S,group", [(4, 4), (3, 5), (12, 4), (40, 7)])
@pytest.mark.parametrize("dim,bits,dt", [(64, 4, "f32"), (128, 4, "f32"), (128, 8, "f16"), (256, 8, "f32")])
def test_rows_behind_a_prefix(S, group, dim, bits, dt):
    print("attention independence", S, group, dim, bits, dt, flush=True)
    heads, page, prefix = 2, 32, 900
    lengths = [1 + 37 * (s % 5) for s in range(S)]
    pages = sum(-(-n // page) for n in lengths) + -(-prefix // page)
    cache = make_cache(pages, heads, page, dim, bits, S)
    tables, rest = tables_of(pages, lengths, page, np.random.default_rng(S))
    q = queries(S, heads * group, dim, dt, S)
    kw = dict(prefix_table=rest, prefix_length=prefix)
    want = check(q, cache, tables, lengths, **kw)
    for other in (30.0, -8.0, 0.0, np.nan):
        # The scores of sequences 1 and 2 many times as large: their references
        # move again and again.  The others' rows are what they were.
        mine = [s for s in range(S) if s not in (1, 2)]
        q2 = q.copy()
        q2[1:3] = (q2[1:3] * other).astype(q.dtype)
        got = host(D.cache_attention(dev(q2), cache[1], dev(tables), dev(np.array(lengths, np.int32)),
                                     prefix_table=dev(rest), prefix_length=dev(np.array([prefix], np.int32)),
                                     out_dtype=torch.float32))
        assert np.array_equal(got[mine], want[mine]), (other, np.argwhere(got[mine] != want[mine])[:4].tolist())
