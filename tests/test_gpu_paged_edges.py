"""The paged operators at the ends of what their arguments may be."""
import pytest
import torch

import tiered_kv_cache_gqa_gb300 as tkv
from test_gpu_paged import BF16, FP16, Pool, close, queries

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("kind,dtype", [("int4", BF16), ("bf16", BF16), ("fp16", FP16)])
@pytest.mark.parametrize("lengths,n", [([3], [6]), ([64], [70]), ([100, 0, 40], [103, 5, 43]), ([700, 2], [1, 9]), ([1200, 33], [8, 60])])
@pytest.mark.parametrize("window", [MOST, MOST - 5, 2 ** 30 + 1])
def test_the_largest_windows_where_queries_come_before_the_first_position(kind, dtype, lengths, n, window):
    """More queries than positions: those before the first see nothing, the others all up to their own, as without a window."""
    p = Pool(kind, lengths, n, page=16).fill()
    q = queries(p, 3, dtype=dtype)
    want = p.oracle(q)
    for max_len in (1, max(lengths), 1 << 30):
        close(p, *p.cache.attend(q, p.cu_t, max_new=max(n), max_len=max_len, window=window, return_lse=True), want, dtype)


@pytest.mark.parametrize("window", [MOST, 2 ** 30 + 7, 2 ** 30, 5])
def test_windows_of_a_sequence_that_counts_more_positions_than_its_table(window):
    """lengths up to 2^31 - 1: the positions beyond the table are left out, and the window counts from the query's own position."""
    p = Pool("int4", [48, 48], [1, 2], page=16).fill()
    q = queries(p, 2)
    for far in (MOST, 2 ** 30 + 40):
        p.lens.fill_(far)
        out, lse = p.cache.attend(q, p.cu_t, window=window, return_lse=True)
        for row, (b, last) in enumerate(((0, far - 1), (1, far - 2), (1, far - 1))):
            first = max(0, last - window + 1)
            if first >= 48:
                assert not out[row].any() and lse[row].isneginf().all()
                continue
            p.lens.fill_(48)                          # the same positions by a query at the table's end and a window back to `first`
            want = p.oracle(q[row:row + 1], 48 - first, cu=[0, 1, 1] if b == 0 else [0, 0, 1])
            p.lens.fill_(far)
            close(p, out[row:row + 1], lse[row:row + 1], want, BF16)


def test_tensors_to_write_to_are_not_overwritten_unnoticed():
    """out, lse, k and v that autograd keeps for a backward pass: the pass says that they have changed."""
    p = Pool("int4", [40], [2], page=16).fill()
    q = queries(p, 2)
    out, lse = torch.randn_like(q), torch.randn(q.shape[:2], device="cuda")
    k, v = (torch.randn(2, 2, 64, device="cuda") for _ in range(2))
    for kept, call in ((out, lambda: p.cache.attend(q, p.cu_t, out=out)), (lse, lambda: p.cache.attend(q, p.cu_t, lse=lse)),
                       (k, lambda: p.cache.gather(p.cu_t, 2, k=k, v=v)), (v, lambda: p.cache.gather(p.cu_t, 2, k=k, v=v))):
        leaf = torch.ones_like(kept).requires_grad_()
        y = (leaf * kept).sum()
        call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()


def test_caches_share_a_workspace():
    """The layers of a model, one after the other on a stream: one workspace for all, as large as the largest call wants it."""
    pools = [Pool("int4", [300 + 7 * i], [1 + i % 3], d=128, page=16, seed=i).fill() for i in range(8)]
    q = [queries(p, 2 + i % 5, seed=i) for i, p in enumerate(pools)]
    outs = [torch.empty_like(x) for x in q]
    size = pools[0].cache._c
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        for p, x, o in zip(pools, q, outs):
            p.cache.attend(x, p.cu_t, out=o, max_new=p.n[0])
        kept = torch.cuda.memory_allocated() - before
        torch.cuda.synchronize()
    assert kept <= tkv.tkv_paged_attention_workspace(size, 12, 3) + (2 << 20)
    for p, x, o in zip(pools, q, outs):
        close(p, o, None, p.oracle(x), BF16)
