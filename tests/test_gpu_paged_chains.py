"""The paged operators behind one another without a pause: what a call reads is what the calls before it wrote."""
import pytest
import torch

import tiered_kv_cache_gqa_gb300 as tkv
from test_gpu_paged import BF16, FP16, Pool, close, ints, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,dtype", [("int4", BF16), ("bf16", BF16), ("fp16", FP16)])
@pytest.mark.parametrize("lengths,max_len", [([180, 37, 250], 250), ([3000, 2000, 700], 3000)])
def test_steps_that_rewrite_what_the_last_ones_read(kind, dtype, lengths, max_len):
    """Every step puts new values where the one before it was read from: the turned q and k, the pages' rows and the rows
    read back.  Only the framework's kernels run in between, so each starts while its predecessors end.  The same steps with
    a wait behind each call give the same bits; attentions of whole items and of cut ones."""
    steps, G, hkv, d = 60, 4, 2, 128
    n = [1, 3, 2]
    p = Pool(kind, lengths, n, hkv=hkv, d=d, page=16).fill()
    rows = sum(n)
    g = torch.Generator("cuda").manual_seed(2)
    qs = torch.randn(steps, rows, hkv * G, d, generator=g, device="cuda").to(dtype)
    ks, vs = (torch.randn(steps, rows, hkv, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    pos = torch.randint(0, 4096, (steps, 2, rows), generator=g, device="cuda", dtype=torch.int32)
    rot = tkv.Rotary(tkv.rope_table(4096, d), [0] * 40 + [1] * 24)
    start = p.pages.clone()

    def run(wait):
        p.pages.copy_(start)
        q, k = torch.empty_like(qs[0]), torch.empty_like(ks[0])
        kk, vv = torch.empty_like(k), torch.empty_like(k)
        outs = torch.zeros(steps, rows, hkv * G, d, device="cuda", dtype=dtype)
        lses, read = torch.zeros(steps, rows, hkv * G, device="cuda"), torch.zeros(steps, 2, rows, hkv, d, device="cuda", dtype=dtype)
        torch.cuda.synchronize()
        none = torch.cuda.synchronize if wait else lambda: None
        for t in range(steps):
            tkv.rope(qs[t], rot, pos[t], out=q)
            none()
            tkv.rope(ks[t], rot, pos[t], out=k)
            none()
            p.cache.append(k, vs[t], p.cu_t)
            none()
            p.cache.gather(p.cu_t, rows, k=kk, v=vv)                     # the rows that the append has just written
            none()
            p.cache.attend(q, p.cu_t, max_new=3, max_len=max_len, out=outs[t], lse=lses[t])
            none()
            p.cache.append(vv, kk, p.cu_t, rotary=rot, positions=pos[t])   # and once more, from what the gather read
            none()
            p.cache.gather(p.cu_t, rows, k=read[t, 0], v=read[t, 1])
            none()
        torch.cuda.synchronize()
        return outs, lses, read, p.pages.clone()

    want = run(True)
    assert want[0].isfinite().all() and not torch.equal(want[0][0], want[0][1])
    for _ in range(3):
        got = run(False)
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    lens = ints(lengths)
    assert torch.equal(p.lens, lens)


@pytest.mark.parametrize("kind,dtype", [("bf16", BF16), ("fp16", FP16), ("int4", BF16)])
@pytest.mark.parametrize("max_len", [256, 4000])
def test_pages_that_are_missing_in_turn(kind, dtype, max_len):
    """Every other page is none, where the ring's slots hold other tiles from before: each tile goes by its own flag."""
    p = Pool(kind, [4000, 1500, 300], [1, 1, 2], d=64, page=16).fill()
    p.pt[:, 1::2] = -1
    p.pt[0, 40:44], p.pt[0, 101] = -1, p.num_pages
    p.table.copy_(torch.tensor(p.pt))
    q, status = queries(p, 4, dtype=dtype), ints([0])
    want = p.oracle(q)
    first = p.cache.attend(q, p.cu_t, max_len=max_len, return_lse=True, status=status)
    assert status.item() == tkv.TKV_ECAPACITY
    close(p, *first, want, dtype)
    for _ in range(30):
        got = p.cache.attend(q, p.cu_t, max_len=max_len, return_lse=True)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
