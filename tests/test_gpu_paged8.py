"""8-bit pages against the fp64 oracle: append with its block scales, gather, attention."""
import numpy as np
import pytest
import torch

import tiered_kv_cache_gqa_gb300 as tkv
from oracle import paged, paged8
from test_gpu_paged import APPENDS, BF16, FP16, FP32, close, f32, ints, queries

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


class Pool8:
    """An 8-bit paged cache on both sides."""
    kind = "e4m3"

    def __init__(self, lengths, n, hkv=2, d=64, page=16, max_pages=None, seed=0, spare=2):
        self.lengths, self.n, self.hkv, self.d, self.page = lengths, n, hkv, d, page
        rng = np.random.default_rng(seed)
        need = [max(1, -(-x // page)) for x in lengths]
        self.max_pages = max_pages or max(need)
        self.num_pages = sum(need) + spare
        order = rng.permutation(self.num_pages)
        self.pt = np.zeros((len(lengths), self.max_pages), np.int32)
        at = 0
        for b, k in enumerate(need):
            k = min(k, self.max_pages)
            self.pt[b, :k] = order[at:at + k]
            at += k
        self.cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.np_pages = rng.integers(0, 256, (self.num_pages, hkv, page // 16, 32 * d + 16)).astype(np.uint8)   # any bytes, exponents too
        self.pages = torch.tensor(self.np_pages).cuda()
        self.table, self.lens, self.cu_t = ints(self.pt), ints(lengths), ints(self.cu)
        self.cache = tkv.PagedCache(self.pages, self.table, self.lens)

    def fill(self, scale=1.0, seed=3):
        """All positions of all sequences, through the append; both sides then hold the same pages."""
        t = int(sum(self.lengths))
        g = torch.Generator("cuda").manual_seed(seed)
        k, v = ((torch.randn(t, self.hkv, self.d, generator=g, device="cuda") * scale).to(BF16) for _ in range(2))
        self.cache.append(k, v, ints(np.concatenate([[0], np.cumsum(self.lengths)])))
        return self.sync_back()

    def sync_back(self):
        self.np_pages = self.pages.cpu().numpy()
        return self

    def oracle(self, q, window=0, scale=None, cu=None):
        return paged8.attend(f32(q).astype(np.float64), self.np_pages, self.pt, self.lengths, self.cu if cu is None else cu, self.page, window, scale)


def same_pages(p, want, d):
    """All bytes but the 8 that are not used, of records that no row touched too."""
    got = p.pages.cpu().numpy()[..., :32 * d + 8]
    differ = np.argwhere(got != want[..., :32 * d + 8])
    assert not len(differ), (len(differ), [(tuple(x), got[tuple(x)], want[tuple(x)]) for x in differ[:8].tolist()])


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("pairs,axes,interleaved", APPENDS + [(8, 1, False), (24, 2, False), (28, 1, True)])
def test_append_writes_its_rows_and_nothing_else(dtype, d, pairs, axes, interleaved):
    """Byte for byte: new blocks, blocks that hold rows already (with any exponents), empty ones, infinities and NaN."""
    p = Pool8([40, 0, 17, 5, 100, 31], [33, 0, 1, 5, 3, 15], d=d, hkv=3)
    rows = int(p.cu[-1]) + 3                                    # three rows behind the last sequence
    g = torch.Generator("cuda").manual_seed(7)
    k = torch.randn(rows, p.hkv, d, generator=g, device="cuda").to(dtype)
    v = torch.randn(rows, p.hkv, d, generator=g, device="cuda").to(dtype) * 0.125
    k[9:25, 0], v[:8, 1] = 0.0, 0.0                             # an empty block, and rows of one
    k[2, 0, 3], v[3, 0, 5], v[4, 1, d - 1], v[33, 2] = INF, NAN, -INF, INF
    k[36:39, 1] = 60000.0 if dtype == FP16 else 3e38             # saturating
    v[40, 2] = 65504.0
    k[41, 1] *= 2.0 ** -20
    want, kr, rot = p.np_pages.copy(), f32(k), None
    pos = torch.randint(0, 900, (axes, rows), generator=g, device="cuda", dtype=torch.int32)
    if pairs:
        table = tkv.rope_table(900, 2 * pairs)
        axis = [j * axes // pairs for j in range(pairs)]
        rot = tkv.Rotary(table, axis, interleaved)
        with np.errstate(all="ignore"):
            kr = paged.rotate(kr, table.cpu().numpy(), pos.cpu().numpy(), axis, interleaved)
    status = ints([0])
    p.cache.append(k, v, p.cu_t, rotary=rot, positions=pos if pairs else None, status=status)
    assert status.item() == 0
    paged8.append(want, p.pt, p.lengths, p.cu, p.page, kr, f32(v))
    same_pages(p, want, d)
    # and back out: rounded once
    for out_t in (BF16, FP16, FP32):
        kk, vv = (torch.full((rows, p.hkv, d), 7.0, device="cuda", dtype=out_t) for _ in range(2))
        p.cache.gather(p.cu_t, rows, k=kk, v=vv)
        assert (kk[int(p.cu[-1]):] == 7).all() and (vv[int(p.cu[-1]):] == 7).all()
        for b, (ln, n) in enumerate(zip(p.lengths, p.n)):
            for h in range(p.hkv if n else 0):
                _, K, V, _ = paged8.sequence(want, p.pt, b, ln, p.page, h)
                for got, x in ((kk, K), (vv, V)):
                    w = torch.tensor(x[ln - n:].astype(np.float32)).to(out_t)
                    got = got[int(p.cu[b]):int(p.cu[b + 1]), h].cpu()
                    assert torch.equal(got.nan_to_num(1.0), w.nan_to_num(1.0)) and torch.equal(got.isnan(), w.isnan())


@pytest.mark.parametrize("d,page,hkv", [(128, 64, 8), (64, 16, 1), (64, 32, 11), (128, 128, 2)])
def test_token_by_token_and_drafts_that_are_taken_back(d, page, hkv):
    """Steps of 1, 2, 5 and 16 rows into the same blocks, rows that grow the scale, lengths that go back after rejected drafts."""
    p = Pool8([0, 0, 0], [1, 1, 1], d=d, page=page, hkv=hkv, max_pages=-(-120 // page), spare=40)
    p.pt = np.arange(p.pt.size, dtype=np.int32).reshape(p.pt.shape)[::-1].copy()
    assert p.pt.max() < p.num_pages
    p.table.copy_(torch.tensor(p.pt))
    rng, want = np.random.default_rng(5), p.np_pages.copy()
    lengths = np.array([0, 3, 9])
    for step in range(24):
        n = rng.choice([1, 1, 2, 5, 16, 0], 3)
        lengths = np.minimum(lengths + n, 120)
        n = np.minimum(n, lengths)
        cu = np.concatenate([[0], np.cumsum(n)])
        if cu[-1] == 0:
            continue
        k, v = ((torch.tensor(rng.standard_normal((int(cu[-1]), hkv, d)) * 2.0 ** rng.integers(-12, 12)).float().to(BF16)) for _ in range(2))
        p.lens.copy_(torch.tensor(lengths.astype(np.int32)))
        p.cache.append(k.cuda(), v.cuda(), ints(cu))
        paged8.append(want, p.pt, lengths, cu, page, f32(k), f32(v))
        if step % 5 == 4:
            lengths = np.maximum(lengths - rng.integers(0, 5, 3), 0)
    same_pages(p, want, d)


def test_append_without_positions_turns_by_the_place_in_the_cache():
    for pairs, interleaved in ((64, False), (32, True), (9, False)):
        a, b = (Pool8([40, 23], [40, 7], d=128, hkv=3) for _ in range(2))
        k, v = (torch.randn(47, 3, 128, device="cuda").to(BF16) for _ in range(2))
        rot = tkv.Rotary(tkv.rope_table(64, 2 * pairs), interleaved=interleaved)
        pos = torch.cat([torch.arange(40), torch.arange(16, 23)]).to(torch.int32).cuda()
        a.cache.append(k, v, a.cu_t, rotary=rot)
        b.cache.append(k, v, b.cu_t, rotary=rot, positions=pos)
        assert torch.equal(a.pages, b.pages)


def test_append_strides_and_a_position_outside_the_table():
    p, q = Pool8([40, 23], [40, 7]), Pool8([40, 23], [40, 7])
    wide = torch.randn(2, 2, 47, 3, 72, device="cuda").to(BF16)
    k, v = wide[0, 0, :, :2, :64], wide[1, 1, :, 1:, 8:]                   # rows and heads apart
    p.cache.append(k, v, p.cu_t)
    q.cache.append(k.contiguous(), v.contiguous(), q.cu_t)
    assert torch.equal(p.pages, q.pages)
    one = k[:, :1].expand(47, 2, 64)                                       # one head for both
    p.cache.append(one, v, p.cu_t)
    q.cache.append(one.contiguous(), v.contiguous(), q.cu_t)
    assert torch.equal(p.pages, q.pages)
    into = torch.full((2, 50, 3, 80), 7.0, device="cuda", dtype=BF16)      # gather into a part of a larger tensor
    p.cache.gather(p.cu_t, 47, k=into[0, :47, 1:, 8:72], v=into[1, 3:, :2, :64])
    kk, vv = p.cache.gather(p.cu_t, 47)
    assert torch.equal(into[0, :47, 1:, 8:72], kk) and torch.equal(into[1, 3:, :2, :64], vv)
    assert (into[0, 47:] == 7).all() and (into[0, :, 0] == 7).all() and (into[1, :3] == 7).all() and (into[1, :, 2] == 7).all()
    status, rot = ints([0]), tkv.Rotary(tkv.rope_table(8, 64))
    pos = ints(list(range(6)) + [8] + [0] * 40)
    p.cache.append(k, v, p.cu_t, rotary=rot, positions=pos, status=status)
    kk, vv = p.cache.gather(p.cu_t, 47)
    assert status.item() == tkv.TKV_EINVAL and kk[6].isnan().all() and kk[:6].isfinite().all() and kk[7:].isfinite().all() and vv.isfinite().all()


def test_rows_without_a_place():
    p = Pool8([20, 50, 3, 33], [2, 20, 5, 1], max_pages=3)      # 50 positions in 48; five rows of three positions
    p.pt[0, 1], p.pt[3, 2] = -1, p.num_pages
    p.table.copy_(torch.tensor(p.pt))
    k, v = (torch.randn(28, 2, 64, device="cuda").to(BF16) for _ in range(2))
    status, want = ints([0]), p.np_pages.copy()
    p.cache.append(k, v, p.cu_t, status=status)
    assert status.item() == tkv.TKV_ECAPACITY
    lost = [i for i in range(28) if paged.row_place(p.cu, p.lengths, p.pt, p.page, p.num_pages, i)[2] is None]
    assert lost == [0, 1, 20, 21, 22, 23, 27]
    paged8.append(want, p.pt, p.lengths, p.cu, p.page, f32(k), f32(v))
    same_pages(p, want, 64)
    for dtype in (FP32, BF16):
        status.zero_()
        kk, vv = p.cache.gather(p.cu_t, 28, dtype=dtype, status=status)
        assert status.item() == tkv.TKV_ECAPACITY and kk[lost].isnan().all() and vv[lost].isnan().all()
        rest = [i for i in range(28) if i not in lost]
        assert kk[rest].isfinite().all() and vv[rest].isfinite().all()


@pytest.mark.parametrize("cu", [[0, 5, 3, 9, 4], [0, 40, 41, 42, 43], [-3, 2, 4, 6, 8], [7, 7, 7, 7, 7], [2 ** 31 - 1, -2 ** 31, 5, 0, 3]])
@pytest.mark.parametrize("lengths", [[20, 50, 3, 33], [-1, 2 ** 31 - 1, -2 ** 31, 5]])
def test_offsets_and_lengths_that_make_no_sense(cu, lengths):
    """Nothing outside the pages and the outputs is touched, and the context stays usable."""
    p = Pool8([20, 50, 3, 33], [2, 20, 5, 1])
    guard = torch.full((64, 2, 64), 7.0, device="cuda", dtype=BF16)
    k, v = guard[8:36], torch.randn(28, 2, 64, device="cuda").to(BF16)
    p.lens.copy_(ints(lengths))
    p.cache.append(k, v, ints(cu), status=ints([0]))
    p.cache.gather(ints(cu), 28, k=guard[8:36], v=torch.empty_like(v), status=ints([0]))
    assert (guard[:8] == 7).all() and (guard[36:] == 7).all()
    p.lens.copy_(ints(p.lengths))
    p.cache.append(v, v, p.cu_t)
    there = [paged.row_place(p.cu, p.lengths, p.pt, p.page, p.num_pages, i)[2] is not None for i in range(28)]   # five rows of three positions
    kk, vv = p.cache.gather(p.cu_t, 28)
    assert sum(there) == 26 and kk[there].isfinite().all() and vv[there].isfinite().all()


def test_many_sequences_and_blocks():
    """More sequences than a search takes in two steps, most of them short, some idle."""
    rng = np.random.default_rng(9)
    lengths = [int(x) for x in rng.integers(0, 30, 1500)]
    n = [int(rng.integers(0, x + 1)) if i % 3 else 0 for i, x in enumerate(lengths)]
    lengths[700], n[700], lengths[1499], n[1499] = 200, 150, 40, 40
    p = Pool8(lengths, n, hkv=1)
    k, v = (torch.randn(int(p.cu[-1]), 1, 64, device="cuda").to(BF16) for _ in range(2))
    want = p.np_pages.copy()
    p.cache.append(k, v, p.cu_t)
    paged8.append(want, p.pt, p.lengths, p.cu, p.page, f32(k), f32(v))
    same_pages(p, want, 64)


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths,n,G,page,window,max_len", [
    ([1], [1], 1, 16, 0, 1), ([0, 1, 16, 17], [1, 1, 1, 1], 8, 16, 0, 40), ([700, 0, 33, 129, 256], [1, 0, 1, 1, 1], 3, 32, 0, 700),
    ([1300], [1], 7, 64, 0, 1300), ([300, 90], [5, 3], 8, 16, 0, 300), ([300, 9, 600], [1, 12, 30], 2, 128, 0, 600),
    ([700, 260, 40], [1, 1, 1], 4, 16, 100, 700), ([700, 260, 40], [4, 1, 7], 5, 16, 33, 700), ([520, 3], [3, 5], 1, 16, 1, 520),
    ([600], [2], 12, 16, 0, 600), ([64, 3], [70, 2], 3, 16, 0, 64)])
def test_attention(dtype, d, lengths, n, G, page, window, max_len):
    p = Pool8(lengths, n, d=d, page=page).fill()
    q = queries(p, G, int(p.cu[-1]) + 2, dtype)
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    p.cache.attend(q, p.cu_t, max_new=max(n), max_len=max_len, window=window, out=out, return_lse=True, lse=lse)
    assert (out[-2:] == 7).all() and (lse[-2:] == 7).all()          # rows behind the last sequence
    want = p.oracle(q, window)
    close(p, out, lse, want, dtype)
    # the estimates choose the split and the tiles, not the result; and the same call gives the same bits
    for new, ln in ((1, 1), (100, 1 << 20), (max(n), 1 << 30)):
        o2, l2 = p.cache.attend(q, p.cu_t, max_new=new, max_len=ln, window=window, return_lse=True)
        close(p, o2, l2, want, dtype)
        o3, l3 = p.cache.attend(q, p.cu_t, max_new=new, max_len=ln, window=window, return_lse=True)
        live = slice(0, int(p.cu[-1]))
        assert torch.equal(o2[live], o3[live]) and torch.equal(l2[live], l3[live])


@pytest.mark.parametrize("d", [64, 128])
def test_attention_of_many_sequences(d):
    """More sequences than threads of a CTA, most of them short, some idle and some empty: the deal of the work, pages that are kept
    for a sequence's heads, the next sequence read ahead."""
    rng = np.random.default_rng(9)
    lengths = [int(x) for x in rng.integers(0, 40, 300)]
    lengths[17], lengths[250] = 3000, 1111
    n = [int(x) for x in rng.integers(0, 4, 300)]
    n[17], n[250] = 1, 3
    p = Pool8(lengths, n, d=d).fill()
    q = queries(p, 4)
    want = p.oracle(q)
    for new, ln in ((1, 3000), (1, 40), (3, 3000), (8, 1 << 30)):
        close(p, *p.cache.attend(q, p.cu_t, max_new=new, max_len=ln, return_lse=True), want, BF16)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths,n,G", [([36007], [1], 3), ([20001, 5], [3, 1], 4), ([2500], [6], 5), ([9000, 0, 41], [1, 1, 1], 8)])
def test_items_of_many_pieces(dtype, d, lengths, n, G):
    """Few long sequences: an item is cut between up to all CTAs, and several of them join it."""
    p = Pool8(lengths, n, d=d, page=64).fill()
    q = queries(p, G, int(p.cu[-1]), dtype)
    want = p.oracle(q)
    for new, ln in ((max(n), max(lengths)), (1, 1 << 20), (100, 1 << 20)):
        out, lse = p.cache.attend(q, p.cu_t, max_new=new, max_len=ln, return_lse=True)
        close(p, out, lse, want, dtype)
        again = p.cache.attend(q, p.cu_t, max_new=new, max_len=ln, return_lse=True)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 3, 8])
def test_blocks_of_very_different_scales(d, new):
    """V from 2^-30 to 2^30 between blocks of one sequence, K too: the weights of a scale apart stay right, and so does their sum."""
    p = Pool8([400, 64], [new, 1], d=d)
    rng = np.random.default_rng(4)
    for spread in (4, 12, 30):
        k, v = (torch.tensor(rng.standard_normal((464, 2, d))).float() for _ in range(2))
        f = torch.tensor(2.0 ** rng.integers(-spread, spread + 1, 29)).float().repeat_interleave(16)[:464, None, None]
        p.cache.append((k * f.clamp(max=4)).to(BF16).cuda(), (v * f.flip(0)).to(BF16).cuda(), ints([0, 400, 464]))
        p.sync_back()
        q = queries(p, 3)
        want = p.oracle(q)
        for ln in (400, 1):
            close(p, *p.cache.attend(q, p.cu_t, max_new=new, max_len=ln, return_lse=True), want, BF16)


def test_pages_of_zeros_and_exponents_that_make_no_sense():
    p = Pool8([100, 40], [1, 1]).fill()
    q = queries(p, 4)
    p.pages.zero_()
    p.sync_back()
    out, lse = p.cache.attend(q, p.cu_t, return_lse=True)
    close(p, out, lse, p.oracle(q), BF16)
    assert not out.any() and torch.allclose(lse[0], torch.full_like(lse[0], float(np.log(100))), atol=1e-5)
    p.fill()
    tail = p.pages[..., 32 * p.d:32 * p.d + 8].contiguous().view(torch.int32)
    for e in (-33, 1000, -2 ** 31, 2 ** 31 - 1):
        tail[:, 0, :, 1] = e                                        # V of head 0
        p.pages[..., 32 * p.d:32 * p.d + 8] = tail.view(torch.uint8)
        p.sync_back()
        close(p, *p.cache.attend(q, p.cu_t, return_lse=True), p.oracle(q), BF16)
        kk, vv = p.cache.gather(ints([0, 100, 140]), 140, dtype=FP32)
        _, _, V, _ = paged8.sequence(p.np_pages, p.pt, 0, 100, p.page, 0)
        assert np.array_equal(vv[:100, 0].cpu().numpy(), V.astype(np.float32))


def test_attention_strides_scale_and_logits_far_apart():
    p = Pool8([900, 77], [2, 1], d=128).fill()
    rows = 3
    wide = torch.randn(rows, 3, 8, 128 + 8, device="cuda").to(BF16)
    q = wide[:, 1, :, :128]
    out = torch.zeros(8, rows, 128, device="cuda", dtype=BF16).transpose(0, 1)
    for scale in (None, 2.0, -0.3, 0.0, 40.0):
        p.cache.attend(q, p.cu_t, out=out, scale=scale)
        close(p, out, None, p.oracle(q, scale=scale), BF16)
    for sign in (1.0, -1.0):
        k = torch.zeros(977, 2, 128, device="cuda")
        k[:, :, 0] = torch.cat([torch.arange(900), torch.arange(77)]).cuda()[:, None] * 0.5 * sign
        p.cache.append(k.to(BF16), torch.randn(977, 2, 128, device="cuda").to(BF16), ints([0, 900, 977]))
        p.sync_back()
        q = torch.ones(rows, 8, 128, device="cuda", dtype=BF16)
        o, l = p.cache.attend(q, p.cu_t, scale=1.0, return_lse=True)
        close(p, o, l, p.oracle(q, scale=1.0), BF16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ln", [150, 1 << 30])
def test_nan_where_a_query_does_not_look(d, ln):
    """A NaN behind the end, before the window and among the step's own later tokens; where a query looks it shows, in its channel."""
    p = Pool8([150, 40], [6, 3], d=d, page=32).fill()
    q = queries(p, 3)
    window = 60
    k, v = p.cache.gather(p.cu_t, 9)
    v[4, 0, 3], k[5, 1, 2], v[8, 1, d - 1] = NAN, INF, INF
    p.cache.append(k, v, p.cu_t)
    p.lens.copy_(ints([80, 0]))                                     # positions 70 .. 79 of sequence 0: before every window
    bad = torch.full((10, 2, d), NAN, device="cuda", dtype=BF16)
    p.cache.append(bad, bad, ints([0, 10, 10]))
    p.lens.copy_(ints([150, 40]))
    p.sync_back()
    got = f32(p.cache.attend(q, p.cu_t, window=window, max_len=ln, max_new=6 if ln < 1000 else 11))
    with np.errstate(all="ignore"):
        want = p.oracle(q, window)[0]
    assert np.isnan(want[4, :3]).any() and not np.isnan(want[:4]).any() and not np.isnan(want[6:8]).any()
    assert np.array_equal(np.isfinite(got), np.isfinite(want))
    some = np.isfinite(want)
    # p's rounding 2^-11 and the sums' 2^-14 of at most max |V| < 6, the result's 2^-8: below 2^-7 (1 + |o|)
    assert np.all(np.abs(got[some] - want[some]) <= 2.0 ** -7 * (1 + np.abs(want[some])))


def test_positions_in_bad_pages_are_left_out():
    p = Pool8([200, 64, 4000], [2, 1, 1], page=32, max_pages=125).fill()
    p.pt[0, 2], p.pt[1, 0], p.pt[2, 1::2] = -7, 2 ** 30, -1
    p.table.copy_(torch.tensor(p.pt))
    p.lengths = [200, 64, 4001]                                           # and one position behind the table
    p.lens.copy_(ints(p.lengths))
    q, status = queries(p, 4), ints([0])
    want = p.oracle(q)
    for ln in (1, 200, 4000):
        status.zero_()
        out, lse = p.cache.attend(q, p.cu_t, max_len=ln, return_lse=True, status=status)
        assert status.item() == tkv.TKV_ECAPACITY
        close(p, out, lse, want, BF16)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 30 + 1])
def test_the_largest_windows(window):
    for lengths, n in (([64], [70]), ([700, 2], [1, 9]), ([1200, 33], [8, 60])):
        p = Pool8(lengths, n).fill()
        q = queries(p, 3)
        want = p.oracle(q)
        for ln in (1, max(lengths), 1 << 30):
            close(p, *p.cache.attend(q, p.cu_t, max_new=max(n), max_len=ln, window=window, return_lse=True), want, BF16)


def test_a_cache_whose_offsets_pass_32_bits():
    """Pages whose bytes lie behind 2^32, and a sequence of 300,000 positions."""
    page, d, hkv = 128, 128, 8
    pages = (1 << 32) // (hkv * (page // 16) * (32 * d + 16)) + 3000
    table = ints([[pages - 1 - i for i in range(2400)]])
    cache = tkv.PagedCache.empty(pages, table, ints([300000]), num_kv_heads=hkv, head_dim=d, page_size=page, dtype="e4m3")
    g = torch.Generator("cuda").manual_seed(1)
    k, v = (torch.randn(20000, hkv, d, generator=g, device="cuda").to(BF16) for _ in range(2))
    cache.append(k, v, ints([0, 20000]))
    kk, vv = cache.gather(ints([0, 20000]), 20000)
    assert torch.equal(kk == 0, (k == 0) | (kk == 0)) and ((kk - k).abs() <= 2.0 ** -4 * k.abs() + 2.0 ** -8).all()
    assert ((vv - v).abs() <= 2.0 ** -4 * v.abs() + 2.0 ** -8).all()
    # the other 280,000 positions are zeros: softmax over them and the new ones, in 64 bits
    q = torch.randn(1, 16, d, generator=g, device="cuda").to(BF16)
    out, lse = cache.attend(q, ints([0, 1]), return_lse=True)
    for h in (0, 9, 15):
        z = (kk[:, h // 2].double() @ q[0, h].double()) / d ** 0.5
        z = torch.cat([torch.zeros(280000, dtype=torch.float64, device="cuda"), z])
        total = torch.logsumexp(z, 0)
        want = torch.exp(z[280000:] - total) @ vv[:, h // 2].double()
        # p to 2^-11 and sums to 2^-14 of sum |w v| < 1, small p: 300,000 * 8 * 2^-30, the result's 2^-9 of itself
        assert ((out[0, h].double() - want).abs() <= 2.0 ** -10 + 3e5 * 8 * 2.0 ** -30 + 2.0 ** -9 * want.abs()).all()
        assert abs(lse[0, h].item() - total.item()) <= 2.0 ** -12


def test_captured_and_replayed_on_other_streams():
    """Append, gather and attend captured together, replayed while lengths grow; two graphs beside each other."""
    def build(seed):
        p = Pool8([300, 40], [2, 1], d=128, hkv=2, max_pages=40, spare=60, seed=seed)
        p.pt = np.arange(80, dtype=np.int32).reshape(2, 40)
        p.table.copy_(torch.tensor(p.pt))
        p.pages.zero_()
        g = torch.Generator("cuda").manual_seed(seed)
        ks, vs = (torch.randn(8, 3, 2, 128, generator=g, device="cuda").to(BF16) for _ in range(2))
        qs = torch.randn(8, 3, 8, 128, generator=g, device="cuda").to(BF16)
        return p, ks, vs, qs

    def step(p, k, v, q, rot):
        p.cache.append(k, v, p.cu_t, rotary=rot)
        back = p.cache.gather(p.cu_t, 3)
        return p.cache.attend(tkv.rope(q, rot, p.pos), p.cu_t, max_new=2, return_lse=True) + back

    rot = tkv.Rotary(tkv.rope_table(1024, 128))
    wants, graphs, outs, ins = [], [], [], []
    for seed in (1, 2):
        p, ks, vs, qs = build(seed)
        p.pos = ints([0, 0, 0])
        want = []
        for t in range(8):
            p.lens.copy_(ints([300 + 2 * t, 40 + t]))
            want.append([x.clone() for x in step(p, ks[t], vs[t], qs[t], rot)])
        wants.append(want)
        p.pages.zero_()
        k, v, q = ks[0].clone(), vs[0].clone(), qs[0].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(p, k, v, q, rot)
        graphs.append(graph)
        outs.append(out)
        ins.append((p, k, v, q, ks, vs, qs))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    torch.cuda.synchronize()
    for t in range(8):
        for i in range(2):
            p, k, v, q, ks, vs, qs = ins[i]
            lens = ints([300 + 2 * t, 40 + t])
            streams[i].wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(streams[i]):
                p.lens.copy_(lens)
                k.copy_(ks[t]), v.copy_(vs[t]), q.copy_(qs[t])
                graphs[i].replay()
                got[i].append([x.clone() for x in outs[i]])
            lens.record_stream(streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(got[i], wants[i]):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("lengths,max_len", [([180, 37, 250], 250), ([3000, 2000, 700], 3000)])
def test_steps_that_rewrite_what_the_last_ones_read(lengths, max_len):
    """Every step puts new values where the one before it was read from, without a pause: the same bits as with a wait behind each call."""
    steps, n, rows = 40, [1, 3, 2], 6
    p = Pool8(lengths, n, d=128).fill()
    g = torch.Generator("cuda").manual_seed(2)
    qs = torch.randn(steps, rows, 8, 128, generator=g, device="cuda").to(BF16)
    ks, vs = (torch.randn(steps, rows, 2, 128, generator=g, device="cuda").to(BF16) for _ in range(2))
    pos = torch.randint(0, 4096, (steps, 2, rows), generator=g, device="cuda", dtype=torch.int32)
    rot = tkv.Rotary(tkv.rope_table(4096, 128), [0] * 40 + [1] * 24)
    start = p.pages.clone()

    def run(none):
        p.pages.copy_(start)
        q, k = torch.empty_like(qs[0]), torch.empty_like(ks[0])
        kk, vv = torch.empty_like(k), torch.empty_like(k)
        outs, lses = torch.zeros(steps, rows, 8, 128, device="cuda", dtype=BF16), torch.zeros(steps, rows, 8, device="cuda")
        read = torch.zeros(steps, 2, rows, 2, 128, device="cuda", dtype=BF16)
        torch.cuda.synchronize()
        for t in range(steps):
            for call in (lambda: tkv.rope(qs[t], rot, pos[t], out=q), lambda: tkv.rope(ks[t], rot, pos[t], out=k), lambda: p.cache.append(k, vs[t], p.cu_t),
                         lambda: p.cache.gather(p.cu_t, rows, k=kk, v=vv),
                         lambda: p.cache.attend(q, p.cu_t, max_new=3, max_len=max_len, out=outs[t], lse=lses[t]),
                         lambda: p.cache.append(vv, kk, p.cu_t, rotary=rot, positions=pos[t]), lambda: p.cache.gather(p.cu_t, rows, k=read[t, 0], v=read[t, 1])):
                call()
                none()
        torch.cuda.synchronize()
        return outs, lses, read, p.pages.clone()

    want = run(torch.cuda.synchronize)
    assert want[0].isfinite().all() and not torch.equal(want[0][0], want[0][1])
    for _ in range(3):
        for a, b in zip(run(lambda: None), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_refusals():
    p = Pool8([40], [2])
    k = torch.zeros(2, 2, 64, device="cuda", dtype=BF16)
    for call in (lambda: tkv.PagedCache(p.pages, p.table, p.lens, k_gain=torch.ones(2, device="cuda")), lambda: tkv.PagedCache(p.pages[..., :2048], p.table, p.lens),
                 lambda: tkv.PagedCache(p.pages.view(torch.int8), p.table, p.lens), lambda: p.cache.append(k.float(), k.float(), p.cu_t),
                 lambda: p.cache.append(k, k.half(), p.cu_t), lambda: p.cache.append(k[:, :1], k[:, :1], p.cu_t), lambda: p.cache.attend(k.float(), p.cu_t),
                 lambda: p.cache.attend(torch.zeros(2, 3, 64, device="cuda", dtype=BF16), p.cu_t), lambda: p.cache.gather(p.cu_t, 2, dtype=torch.uint8),
                 lambda: tkv.PagedCache.empty(2, p.table, p.lens, num_kv_heads=2, head_dim=96, page_size=16, dtype="e4m3")):
        with pytest.raises(tkv.TkvError) as e:
            call()
        assert e.value.status == tkv.TKV_EINVAL
    empty = tkv.PagedCache.empty(3, p.table, p.lens, num_kv_heads=2, head_dim=128, page_size=32, dtype="e4m3")
    assert empty.pages.shape == (3, 2, 2, 32 * 128 + 16) and not empty.is_int4
    assert p.cache.attend(k[:0], p.cu_t).shape == (0, 2, 64)
