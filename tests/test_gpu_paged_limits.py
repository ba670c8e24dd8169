"""Attention steps of as many tiles as a step may have."""
import pytest
import torch

import tiered_kv_cache_gqa_gb300 as tkv
from test_gpu_paged import BF16, FP16, Pool, close, ints, queries
from test_gpu_paged8 import Pool8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,d,dtype,positions", [("e4m3", 128, BF16, 16), ("e4m3", 64, FP16, 32), ("int4", 128, BF16, 32), ("int4", 64, FP16, 32),
                                                  ("bf16", 128, BF16, 16), ("fp16", 64, FP16, 16)])
@pytest.mark.parametrize("page,length", [(16, 13), (512, 500)])
def test_as_many_tiles_as_a_step_may_have(kind, d, dtype, positions, page, length):
    """A million sequences or two, of which two have positions and one a query: (1 / 8 + batch) Hkv tiles(page) is as much as 2 * 10^9 allows, and
    a KV head more is refused.  The attention is that of the two sequences alone."""
    batch, tiles = 1_000_000 if page == 512 else 2_000_000, -(-page // positions)
    hkv = int(2e9 / ((batch + 0.125) * tiles))
    p = (Pool8([length, 5], [1, 0], hkv, d, page) if kind == "e4m3" else Pool(kind, [length, 5], [1, 0], hkv, d, page, gains=False)).fill()
    q = queries(p, 1, dtype=dtype)
    want = p.oracle(q)

    def spread(pages):
        table, lengths, cu = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (batch, batch, batch + 1))
        at = ints([batch // 3, batch - 1]).long()
        table[at], lengths[at] = p.table[:, 0], p.lens
        cu[batch // 3 + 1:] = 1
        return tkv.PagedCache(pages, table[:, None], lengths), cu

    cache, cu = spread(p.pages)
    for max_len in (None, 3, 100000):                    # estimates of one length, of short and of long sequences
        status = ints([0])
        close(p, *cache.attend(q, cu, max_len=max_len, return_lse=True, status=status), want, dtype)
        assert status.item() == 0
    more = torch.zeros(p.num_pages, hkv + 1, *p.pages.shape[2:], dtype=p.pages.dtype, device="cuda")
    cache, cu = spread(more)
    with pytest.raises(tkv.TkvError) as e:
        cache.attend(torch.zeros(1, hkv + 1, d, dtype=dtype, device="cuda"), cu)
    assert e.value.status == tkv.TKV_EINVAL
