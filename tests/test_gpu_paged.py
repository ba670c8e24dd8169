"""The operators around a paged cache against the fp64 oracle: rotation, append, gather, attention, and a run of them."""
import math

import numpy as np
import pytest
import torch

import tiered_kv_cache_gqa_gb300 as tkv
from oracle import paged

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def f32(x):
    return x.float().cpu().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check_rotation(y, x, table, pos, axis, interleaved, inverse):
    """y against the exact rotation: three fp32 roundings of at most |x0| + |x1|, one to y's type."""
    x64, t = f32(x).astype(np.float64), table.cpu().numpy().astype(np.float64)
    want, mag = x64.copy(), np.zeros_like(x64)
    n = t.shape[1]
    for j in range(n):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + n)
        c, s = (t[pos[axis[j]], j, i][:, None] for i in (0, 1))
        s = -s if inverse else s
        want[:, :, a], want[:, :, b] = x64[:, :, a] * c - x64[:, :, b] * s, x64[:, :, b] * c + x64[:, :, a] * s
        mag[:, :, a] = mag[:, :, b] = np.abs(x64[:, :, a]) + np.abs(x64[:, :, b])
    tiny = torch.finfo(y.dtype).tiny * torch.finfo(y.dtype).eps
    tol = 3 * 2.0 ** -24 * mag + (0 if y.dtype == FP32 else half_step(y.dtype) * (np.abs(want) + 3 * 2.0 ** -24 * mag)) + tiny
    tol[:, :, 2 * n:] = 0
    assert np.all(np.abs(f32(y) - want) <= tol)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("rows,heads,d,pairs,axes,interleaved", [
    (1, 1, 128, 64, 1, False), (3, 28, 128, 64, 1, False), (1, 1, 2, 1, 1, True), (7, 5, 80, 28, 2, True), (7, 5, 80, 24, 3, False),
    (130, 3, 64, 20, 4, False), (33, 64, 64, 32, 3, True), (2, 3, 18, 9, 1, False), (5, 2, 514, 256, 2, False), (257, 9, 96, 16, 1, True)])
def test_rope(dtype, rows, heads, d, pairs, axes, interleaved):
    g = torch.Generator("cuda").manual_seed(rows + d)
    x = torch.randn(rows, heads, d, generator=g, device="cuda").to(dtype)
    table = tkv.rope_table(100003, 2 * pairs)
    pos = torch.randint(0, 100003, (axes, rows), generator=g, device="cuda", dtype=torch.int32)
    axis = [j * axes // pairs if pairs >= axes else 0 for j in range(pairs)]
    rot = tkv.Rotary(table, axis, interleaved)
    p = pos.cpu().numpy()
    for inverse in (False, True):
        y = tkv.rope(x, rot, pos, inverse=inverse)
        check_rotation(y, x, table, p, axis, interleaved, inverse)
        z = x.clone()
        assert tkv.rope(z, rot, pos, out=z, inverse=inverse) is z and torch.equal(z, y)   # in place


def test_rope_strides_broadcast_and_alignment():
    g = torch.Generator("cuda").manual_seed(5)
    table, n = tkv.rope_table(64, 64), 11
    rot, pos = tkv.Rotary(table), torch.arange(n, device="cuda", dtype=torch.int32)
    base = torch.randn(4, n, 3 * 64 + 8, generator=g, device="cuda").to(BF16)
    x = base[:, :, 1:193].unflatten(2, (3, 64))[1]                 # rows of odd alignment
    want = tkv.rope(x.contiguous(), rot, pos)
    assert torch.equal(tkv.rope(x, rot, pos), want)
    heads_first = x.transpose(0, 1).contiguous().transpose(0, 1)     # [T, H, d] over [H, T, d]
    out = torch.full((3, n, 64), 7.0, device="cuda", dtype=BF16).transpose(0, 1)
    assert torch.equal(tkv.rope(heads_first, rot, pos, out=out), want)
    one = x[:, :1].expand(n, 5, 64)                                  # one head broadcast to five
    assert torch.equal(tkv.rope(one, rot, pos), want[:, :1].expand(n, 5, 64))
    into = torch.full((n, 4, 66), 7.0, device="cuda", dtype=BF16)    # a part of a larger tensor: the rest stays
    tkv.rope(x, rot, pos, out=into[:, 1:, 1:65])
    assert torch.equal(into[:, 1:, 1:65], want) and (into[:, 0] == 7).all() and (into[:, :, 65] == 7).all() and (into[:, :, 0] == 7).all()


def test_rope_gradient_by_differences():
    """The inverse is the gradient: sum(w * rope(x + h e) - w * rope(x)) / h, in fp32 with h = 1 (the map is linear)."""
    g = torch.Generator("cuda").manual_seed(6)
    x, w = (torch.randn(3, 2, 24, generator=g, device="cuda") for _ in range(2))
    rot = tkv.Rotary(tkv.rope_table(50, 20), [0] * 4 + [1] * 6, True)
    pos = torch.randint(0, 50, (2, 3), generator=g, device="cuda", dtype=torch.int32)
    grad = tkv.rope(w, rot, pos, inverse=True)
    y = tkv.rope(x, rot, pos).double()
    for i in range(0, x.numel(), 5):
        e = x.clone().view(-1)
        e[i] += 1.0
        diff = (w.double() * (tkv.rope(e.view_as(x), rot, pos).double() - y)).sum().item()
        # two results and x + h, each rounded to 2^-24 of values below 8; |w| < 8
        assert abs(diff - grad.view(-1)[i].item()) <= 2 * 8 * 4 * 8 * 2.0 ** -24


def test_rope_position_outside_the_table():
    rot, status = tkv.Rotary(tkv.rope_table(8, 16), [0, 0, 0, 0, 1, 1, 1, 1]), ints([0])
    x = torch.ones(3, 2, 16, device="cuda")
    for bad in (8, -1, 2 ** 31 - 1, -2 ** 31):
        status.zero_()
        y = tkv.rope(x, rot, ints([[0, 1, 2], [3, bad, 4]]), status=status)
        assert status.item() == tkv.TKV_EINVAL and y[1, :, 4:8].isnan().all() and y[1, :, 12:].isnan().all()
        assert y[[0, 2]].isfinite().all() and y[1, :, :4].isfinite().all()


# ------------------------------------------------------------------ pages
class Pool:
    """A paged cache on both sides."""

    def __init__(self, kind, lengths, n, hkv=2, d=64, page=16, max_pages=None, gains=True, seed=0, spare=2):
        self.kind, self.lengths, self.n, self.hkv, self.d, self.page = kind, lengths, n, hkv, d, page
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
        self.kg = self.vg = None
        if kind == "int4":
            pages = rng.integers(0, 256, (self.num_pages, hkv, page // 16, 18 * d)).astype(np.uint8)   # any bytes, NaN scales too
            if gains:
                self.kg, self.vg = (rng.uniform(0.001, 0.02, hkv).astype(np.float32) for _ in range(2))
        else:
            pages = np.full((self.num_pages, hkv, 2, page, d), np.nan, np.float32)
        self.np_pages = pages
        t = torch.tensor(pages).cuda()
        self.pages = t if kind == "int4" else t.to({"bf16": BF16, "fp16": FP16}[kind])
        g = [None if x is None else torch.tensor(x).cuda() for x in (self.kg, self.vg)]
        self.table, self.lens = ints(self.pt), ints(lengths)
        self.cache = tkv.PagedCache(self.pages, self.table, self.lens, *g)
        self.cu_t = ints(self.cu)
        self.rng = rng

    def fill(self, scale=1.0):
        """All positions of all sequences, through the append; both sides then hold the same pages."""
        cu = ints(np.concatenate([[0], np.cumsum(self.lengths)]))
        t = int(sum(self.lengths))
        g = torch.Generator("cuda").manual_seed(3)
        dt = FP16 if self.kind == "fp16" else BF16
        k, v = ((torch.randn(t, self.hkv, self.d, generator=g, device="cuda") * scale).to(dt) for _ in range(2))
        self.cache.append(k, v, cu)
        return self.sync_back()

    def sync_back(self):
        self.np_pages = self.pages.cpu().numpy() if self.kind == "int4" else self.pages.float().cpu().numpy()
        return self

    def oracle(self, q, window=0, scale=None, cu=None, lengths=None):
        return paged.attend(f32(q).astype(np.float64), self.np_pages, self.pt, self.lengths if lengths is None else lengths,
                            self.cu if cu is None else cu, self.page, self.hkv, window, scale, self.kg, self.vg)


APPENDS = [  # pairs, axes, interleaved: halves of whole blocks, adjacent pairs, and what is neither
    (None, 1, False), (32, 1, False), (32, 3, False), (32, 1, True), (16, 2, True), (16, 1, False), (9, 2, False), (13, 1, True), (1, 1, False)]


@pytest.mark.parametrize("kind,dtype", [("int4", BF16), ("int4", FP16), ("bf16", BF16), ("fp16", FP16)])
@pytest.mark.parametrize("pairs,axes,interleaved", APPENDS)
def test_append_writes_its_rows_and_nothing_else(kind, dtype, pairs, axes, interleaved):
    p = Pool(kind, [40, 0, 17, 5], [33, 0, 1, 5], page=16, gains=pairs != 16)
    rows = int(p.cu[-1]) + 3                                    # three rows behind the last sequence
    g = torch.Generator("cuda").manual_seed(7)
    k = torch.randn(rows, p.hkv, p.d, generator=g, device="cuda").to(dtype)
    v = torch.randn(rows, p.hkv, p.d, generator=g, device="cuda").to(dtype) * 0.125
    k[0, 0, :16], v[1, 1, 16:32] = 0.0, 0.0                     # empty blocks
    k[2, 0, 3], v[3, 0, 5], v[4, 1, 63] = float("inf"), float("nan"), -float("inf")
    k[5, 1] = 60000.0 if dtype == FP16 else 3e38                 # saturating scales
    before = p.pages.clone()
    rot, kr = None, f32(k)
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
    want = before.cpu()
    for row in range(rows):
        where = paged.row_place(p.cu, p.lengths, p.pt, p.page, p.num_pages, row)
        if where is None:
            continue
        _, _, pg, off = where
        for h in range(p.hkv):
            if kind == "int4":
                rec = want[pg, h, off // 16].numpy()
                for which, x, gain in ((0, kr[row, h], p.kg), (1, f32(v)[row, h], p.vg)):
                    paged.put(rec, off % 16, which, *paged.quantise(x, 1.0 if gain is None else gain[h]), p.d)
            else:
                want[pg, h, 0, off] = torch.tensor(kr[row, h]).to(dtype)
                want[pg, h, 1, off] = v[row, h].cpu()
    got = p.pages.cpu()
    if kind == "int4":
        assert torch.equal(got, want)
    else:
        assert torch.equal(got.view(torch.int16)[~want.isnan()], want.view(torch.int16)[~want.isnan()])
        assert torch.equal(got.isnan(), want.isnan())
    # and back out: the last rows of each sequence, rounded once
    for out_t in (BF16, FP16, FP32):
        kk, vv = (torch.full((rows, p.hkv, p.d), 7.0, device="cuda", dtype=out_t) for _ in range(2))
        p.cache.gather(p.cu_t, rows, k=kk, v=vv)
        p.sync_back()
        for row in range(rows):
            where = paged.row_place(p.cu, p.lengths, p.pt, p.page, p.num_pages, row)
            if where is None:
                assert (kk[row] == 7).all() and (vv[row] == 7).all()
                continue
            for h in range(p.hkv):
                for got, x in zip((kk, vv), paged.read(p.np_pages, where[2], where[3], h, p.d, p.kg, p.vg)):
                    with np.errstate(over="ignore"):
                        w = torch.tensor(x.astype(np.float32)).to(out_t)   # fp64 products of 8 and 24 bits: one rounding to fp32
                    assert torch.equal(got[row, h].cpu().nan_to_num(1.0), w.nan_to_num(1.0)) and torch.equal(got[row, h].cpu().isnan(), w.isnan())


def test_append_without_positions_turns_by_the_place_in_the_cache():
    p = Pool("bf16", [40, 23], [40, 7], d=128, hkv=3)
    k, v = (torch.randn(47, 3, 128, device="cuda").to(BF16) for _ in range(2))
    rot = tkv.Rotary(tkv.rope_table(64, 128))
    p.cache.append(k, v, p.cu_t, rotary=rot)
    a = p.pages.clone()
    pos = torch.cat([torch.arange(40), torch.arange(16, 23)]).to(torch.int32).cuda()
    p.cache.append(k, v, p.cu_t, rotary=rot, positions=pos)
    assert torch.equal(a.nan_to_num(9.0), p.pages.nan_to_num(9.0))
    kk, vv = p.cache.gather(p.cu_t, 47)
    assert torch.equal(kk, tkv.rope(k, rot, pos)) and torch.equal(vv, v)   # the same rotation, bit for bit


@pytest.mark.parametrize("kind", ["int4", "bf16"])
def test_rows_without_a_place(kind):
    p = Pool(kind, [20, 50, 3, 33], [2, 20, 5, 1], max_pages=3)      # 50 positions in 48; five rows of three positions
    p.pt[0, 1], p.pt[3, 2] = -1, p.num_pages
    p.table.copy_(torch.tensor(p.pt))
    k, v = (torch.randn(28, 2, 64, device="cuda").to(BF16) for _ in range(2))
    before, status = p.pages.clone(), ints([0])
    p.cache.append(k, v, p.cu_t, status=status)
    assert status.item() == tkv.TKV_ECAPACITY
    lost = [i for i in range(28) if paged.row_place(p.cu, p.lengths, p.pt, p.page, p.num_pages, i)[2] is None]
    assert lost == [0, 1, 20, 21, 22, 23, 27]
    status.zero_()
    kk, vv = p.cache.gather(p.cu_t, 28, dtype=FP32, status=status)
    assert status.item() == tkv.TKV_ECAPACITY
    assert kk[lost].isnan().all() and vv[lost].isnan().all()
    rest = [i for i in range(28) if i not in lost]
    assert kk[rest].isfinite().all() and vv[rest].isfinite().all()
    changed = (before != p.pages).flatten(1).any(1) if kind == "int4" else ~p.pages.isnan().flatten(1).all(1)
    assert set(changed.nonzero().flatten().tolist()) <= {int(p.pt[1, i]) for i in range(3)} | {int(p.pt[2, 0])}


# ------------------------------------------------------------------ attention
def close(p, out, lse, want, dtype):
    """out, lse against the oracle, row by row.

    delta: of a logit, whose products are exact and summed in fp32: d + 2 roundings of 2^-23 (the tensor core may
    truncate) of S, the sum of |q k|.  p: delta, the rounding u of its 16-bit form (fp16 2^-11; bf16 in two parts 2^-16),
    ex2's 2^-22 and the sums' rounding, 2^-23 for each of the few hundred partial sums, taken as 2^-14.  All of them
    relative to the sum of alpha |v|.  A small p has an absolute error too: fp16's smallest step is 2^-24, half of it
    2^-25, and the largest p of a row is 2^5 or more (its reference lies at least 5 below its maximum), so each of the
    N positions may be 2^-30 of the row's weight off (bf16: nothing above 2^-120).  Then out's own half step."""
    o64, l64, absv, big, far = want
    live = ~np.isnan(o64[..., 0])
    delta = (p.d + 2) * 2.0 ** -23 * big
    u = 2.0 ** -16 if p.kind == "bf16" else 2.0 ** -11
    tol = (2 * delta[..., None] + u + 2.0 ** -14) * absv + 2.0 ** (-120 if p.kind == "bf16" else -30) * far[..., None]
    tol = tol + half_step(dtype) * (np.abs(o64) + tol) + torch.finfo(dtype).tiny
    err = np.abs(f32(out) - o64)
    assert np.all(err[live] <= tol[live]), "worst %g" % np.max((err / tol)[live])
    if lse is not None:
        ll = lse.cpu().numpy().astype(np.float64)
        none = np.isneginf(l64)
        assert np.array_equal(np.isneginf(ll)[live], none[live])
        some = live & ~none
        assert np.all(np.abs(ll[some] - l64[some]) <= (delta + 2.0 ** -14 + 2.0 ** -22 * np.abs(l64))[some])
        assert not f32(out)[live & none].any()


def queries(p, G, rows=None, dtype=BF16, seed=11):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(rows or int(p.cu[-1]), p.hkv * G, p.d, generator=g, device="cuda").to(dtype)


KINDS = [("int4", BF16), ("int4", FP16), ("bf16", BF16), ("fp16", FP16)]


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths,n,G,page,window,max_len", [
    ([1], [1], 1, 16, 0, 1), ([0, 1, 16, 17], [1, 1, 1, 1], 8, 16, 0, 40), ([700, 0, 33, 129, 256], [1, 0, 1, 1, 1], 3, 32, 0, 700),
    ([1300], [1], 7, 64, 0, 1300), ([300, 90], [5, 3], 8, 16, 0, 300), ([300, 9, 600], [1, 12, 30], 2, 128, 0, 600),
    ([700, 260, 40], [1, 1, 1], 4, 16, 100, 700), ([700, 260, 40], [4, 1, 7], 5, 16, 33, 700), ([520, 3], [3, 5], 1, 16, 1, 520),
    ([600], [2], 12, 16, 0, 600)])
def test_attention(kind, dtype, d, lengths, n, G, page, window, max_len):
    p = Pool(kind, lengths, n, d=d, page=page).fill()
    q = queries(p, G, int(p.cu[-1]) + 2, dtype)
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    p.cache.attend(q, p.cu_t, max_new=max(n), max_len=max_len, window=window, out=out, return_lse=True, lse=lse)
    assert (out[-2:] == 7).all() and (lse[-2:] == 7).all()          # rows behind the last sequence
    want = p.oracle(q, window)
    close(p, out, lse, want, dtype)
    # the estimates choose the split, not the result; and the same call gives the same bits
    for new, ln in ((1, 1), (100, 1 << 20)):
        o2, l2 = p.cache.attend(q, p.cu_t, max_new=new, max_len=ln, window=window, return_lse=True)
        close(p, o2, l2, want, dtype)
        o3, l3 = p.cache.attend(q, p.cu_t, max_new=new, max_len=ln, window=window, return_lse=True)
        live = slice(0, int(p.cu[-1]))
        assert torch.equal(o2[live], o3[live]) and torch.equal(l2[live], l3[live])


@pytest.mark.parametrize("kind,dtype", KINDS)
def test_attention_of_many_sequences(kind, dtype):
    """More sequences than threads of a CTA, most of them short, some idle: the deal of the work."""
    rng = np.random.default_rng(9)
    lengths = [int(x) for x in rng.integers(0, 40, 300)]
    lengths[17], lengths[250] = 3000, 1111
    n = [int(x) for x in rng.integers(0, 2, 300)]
    n[17] = n[250] = 1
    p = Pool(kind, lengths, n, page=16).fill()
    q = queries(p, 4, dtype=dtype)
    want = p.oracle(q)
    for ln in (3000, 40):
        close(p, *p.cache.attend(q, p.cu_t, max_new=1, max_len=ln, return_lse=True), want, dtype)


def test_attention_strides_scale_and_logits_far_apart():
    p = Pool("int4", [900, 77], [2, 1], d=128, page=16).fill()
    G, rows = 4, 3
    wide = torch.randn(rows, 3, 8, 128 + 8, device="cuda").to(BF16)
    q = wide[:, 1, :, :128]
    out = torch.zeros(8, rows, 128, device="cuda", dtype=BF16).transpose(0, 1)
    for scale in (None, 2.0, -0.3, 0.0, 40.0):
        p.cache.attend(q, p.cu_t, out=out, scale=scale)
        close(p, out, None, p.oracle(q, scale=scale), BF16)
    # logits that rise along the sequence, so that the reference has to move often, and fall
    for sign in (1.0, -1.0):
        k = torch.zeros(977, 2, 128, device="cuda")
        k[:, :, 0] = torch.cat([torch.arange(900), torch.arange(77)]).cuda()[:, None] * 0.5 * sign
        p.cache.append(k.to(BF16), torch.randn(977, 2, 128, device="cuda").to(BF16), ints([0, 900, 977]))
        p.sync_back()
        q = torch.ones(rows, 8, 128, device="cuda", dtype=BF16)
        o, l = p.cache.attend(q, p.cu_t, scale=1.0, return_lse=True)
        close(p, o, l, p.oracle(q, scale=1.0), BF16)
    assert p.cache.attend(q.expand(rows, 8, 128), p.cu_t).shape == q.shape


@pytest.mark.parametrize("kind", ["int4", "bf16"])
def test_queries_of_any_size(kind):
    """Rows of q from the smallest to the largest numbers of their type: 4-bit keys meet them scaled."""
    p = Pool(kind, [200], [4], d=64, page=16).fill()
    q = torch.randn(4, 4, 64, device="cuda")
    for i, s in enumerate((1e-30, 1e-5, 1e3, 1e30)):
        q[i] *= s
    q[1, 1] = 0.0
    q = q.to(BF16)
    # logits of 1e30 leave one position per row: the largest
    out, lse = p.cache.attend(q, p.cu_t, return_lse=True)
    want = p.oracle(q)
    o64 = want[0]
    close(p, out[:3], lse[:3], tuple(x[:3] for x in want), BF16)
    assert np.all(np.abs(f32(out[3]) - o64[3]) <= 2.0 ** -8 * np.abs(o64[3]) + 1e-6)
    q[0, 0, 5], q[2, 3, 9] = float("nan"), float("inf")               # a bad row stays alone
    bad, _ = p.cache.attend(q, p.cu_t, return_lse=True)
    assert bad[0, 0].isnan().all() and bad[2, 3].isnan().all()
    keep = torch.ones(4, 4, dtype=torch.bool, device="cuda")
    keep[0, 0] = keep[2, 3] = False
    assert torch.equal(bad[keep], out[keep])


@pytest.mark.parametrize("kind", ["int4", "bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_and_infinity_where_a_query_does_not_look(kind, d):
    """A position that a query does not see may hold anything: in V and in K, behind the end, before the window, and
    among the step's own later tokens; where a query looks, the NaN shows in the channels of its block."""
    dt = FP16 if kind == "fp16" else BF16
    p = Pool(kind, [150, 40], [6, 3], d=d, page=32).fill()
    q = queries(p, 3, dtype=dt)
    window = 60
    k, v = (torch.randn(9, 2, d, device="cuda").to(dt) for _ in range(2))
    k0, v0 = p.cache.gather(p.cu_t, 9, dtype=dt)
    v[:], k[:] = v0, k0
    v[4, 0, 3] = float("nan")          # sequence 0, query 4 (position 148)
    k[5, 1, 2] = float("inf")          # sequence 0, query 5 (149)
    v[8, 1, d - 1] = float("inf")      # sequence 1, query 2
    p.cache.append(k, v, p.cu_t)
    old = ints([80, 0])                # positions 70 .. 79 of sequence 0: before every window, inside its first tile
    p.lens.copy_(old)
    bad = torch.full((10, 2, d), float("nan"), device="cuda", dtype=dt)
    p.cache.append(bad, bad, ints([0, 10, 10]))
    p.lens.copy_(ints([150, 40]))
    p.sync_back()
    got = p.cache.attend(q, p.cu_t, window=window)
    with np.errstate(all="ignore"):
        want = p.oracle(q, window)[0]
    assert np.isnan(want[4, :3]).any() and not np.isnan(want[:4]).any() and not np.isnan(want[6:8]).any()
    assert np.array_equal(np.isfinite(f32(got)), np.isfinite(want))
    some = np.isfinite(want)
    assert np.all(np.abs(f32(got)[some] - want[some]) <= 0.02 * (1 + np.abs(want[some])))


@pytest.mark.parametrize("kind", ["int4", "bf16"])
def test_positions_in_bad_pages_are_left_out(kind):
    p = Pool(kind, [200, 64], [2, 1], page=32, max_pages=5).fill()      # 200 positions, room for 160
    p.pt[0, 2], p.pt[1, 0] = -7, 2 ** 30
    p.table.copy_(torch.tensor(p.pt))
    q, status = queries(p, 4), ints([0])
    for ln in (1, 200):
        status.zero_()
        out, lse = p.cache.attend(q, p.cu_t, max_len=ln, return_lse=True, status=status)
        assert status.item() == tkv.TKV_ECAPACITY
        close(p, out, lse, p.oracle(q), BF16)
    p.pt[1, 1] = -1                                                       # nothing left of sequence 1
    p.table.copy_(torch.tensor(p.pt))
    out, lse = p.cache.attend(q, p.cu_t, return_lse=True)
    assert not out[2].any() and lse[2].isneginf().all()


@pytest.mark.parametrize("kind", ["int4", "bf16"])
def test_lengths_and_offsets_that_make_no_sense(kind):
    """Nothing outside the buffers is touched, whatever the device arrays hold; what has no rows stays as it was."""
    p = Pool(kind, [100, 60], [1, 1], page=16).fill()
    q = queries(p, 2, 4)
    k = torch.randn(4, 2, 64, device="cuda").to(BF16)
    for lens, cu in (([-5, 60], [0, 1, 2]), ([2 ** 31 - 1, -2 ** 31], [0, 1, 2]), ([100, 60], [2, 1, 0]), ([100, 60], [-9, 1, 90]),
                     ([100, 60], [0, 2 ** 31 - 1, -2 ** 31]), ([100, 60], [0, 0, 0]), ([0, 0], [0, 2, 4])):
        p.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        cu = ints(cu)
        status = ints([0])
        for ln in (1, 1000):
            p.cache.attend(q, cu, max_len=ln, status=status)
        p.cache.append(k, k, cu, status=status)
        p.cache.gather(cu, 4, status=status)
    torch.cuda.synchronize()
    p.lens.copy_(ints([100, 60]))
    p.sync_back()
    close(p, *p.cache.attend(q, p.cu_t, return_lse=True), p.oracle(q), BF16)


def test_far_positions_and_pages():
    """Byte offsets beyond 32 bits, in the page pool and in the page table's reach."""
    hkv, d, page = 8, 128, 256
    num_pages = (5 << 30) // (hkv * page * d * 4) + 1                      # 5 GiB of 16-bit pages
    pages = torch.zeros(num_pages, hkv, 2, page, d, dtype=BF16, device="cuda")
    table, lens = ints([[num_pages - 1, num_pages - 2]]), ints([300])
    cache = tkv.PagedCache(pages, table, lens)
    k, v = (torch.randn(300, hkv, d, device="cuda").to(BF16) for _ in range(2))
    cache.append(k, v, ints([0, 300]))
    assert torch.equal(pages[-1, :, 0].transpose(0, 1), k[:256]) and torch.equal(pages[-2, :, 1, :44].transpose(0, 1), v[256:])
    q = torch.randn(1, hkv, d, device="cuda").to(BF16)
    out = cache.attend(q, ints([0, 1])).double()
    z = torch.einsum("hd,thd->ht", q[0].double(), k.double()) / math.sqrt(d)
    want = torch.einsum("ht,thd->hd", z.softmax(-1), v.double())
    assert (out[0] - want).abs().max().item() <= 2.0 ** -8 * want.abs().max().item() + 2.0 ** -12
    del pages, cache
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ how they are used together
@pytest.mark.parametrize("kind,dtype", [("int4", BF16), ("bf16", BF16), ("int4", FP16)])
def test_decode_steps_of_a_layer(kind, dtype):
    """Prompts enter, then steps of one and of several tokens: rotate q, append with rotation, attend; the steps again
    as one captured graph give the same bits."""
    lengths, G, hkv, d = [37, 5, 90], 4, 2, 128
    p = Pool(kind, [64, 48, 112], [0, 0, 0], hkv=hkv, d=d, page=16)
    rot = tkv.Rotary(tkv.rope_table(4096, d), [0] * 24 + [1] * 20 + [2] * 20)
    g = torch.Generator("cuda").manual_seed(1)

    def step_inputs(n):
        t = sum(n)
        return (torch.randn(t, hkv * G, d, generator=g, device="cuda").to(dtype), torch.randn(t, hkv, d, generator=g, device="cuda").to(dtype),
                torch.randn(t, hkv, d, generator=g, device="cuda").to(dtype), torch.randint(0, 4096, (3, t), generator=g, device="cuda", dtype=torch.int32),
                ints(np.concatenate([[0], np.cumsum(n)])))

    def step(q, k, v, pos, cu, n):
        qr = tkv.rope(q, rot, pos)
        p.cache.append(k, v, cu, rotary=rot, positions=pos)
        return qr, p.cache.attend(qr, cu, max_new=max(n), return_lse=True)

    p.lens.zero_()
    for n in (lengths, [1, 1, 1], [3, 0, 2], [1, 4, 1], [1, 1, 1]):
        ins = step_inputs(n)
        p.lens.add_(ints(n))
        qr, (out, lse) = step(*ins, n)
        p.sync_back()
        close(p, out, lse, p.oracle(qr, cu=ins[4].cpu().numpy(), lengths=p.lens.cpu().numpy()), dtype)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, captured = step(*ins, n)
    for x in captured:
        x.zero_()
    p.pages.zero_() if kind != "int4" else None
    if kind != "int4":
        p.pages.copy_(torch.tensor(p.np_pages).to(p.pages.dtype))
    graph.replay()
    assert torch.equal(captured[0], out) and torch.equal(captured[1], lse)
    other = step_inputs(n)                                               # new contents in the same tensors, one position on
    for a, b in zip(ins[:4], other[:4]):
        a.copy_(b)
    p.lens.add_(1)
    graph.replay()
    p.sync_back()
    qr = tkv.rope(ins[0], rot, ins[3])
    close(p, *captured, p.oracle(qr, cu=ins[4].cpu().numpy(), lengths=p.lens.cpu().numpy()), dtype)


def test_partial_results_join_by_lse():
    """Two caches' results, joined by their lse, are the attention over both."""
    a, b = Pool("int4", [300], [1], page=16, seed=1).fill(), Pool("bf16", [500], [1], page=16, seed=2).fill(2.0)
    q = queries(a, 4)
    parts = [x.cache.attend(q, x.cu_t, return_lse=True) for x in (a, b)]
    top = torch.maximum(parts[0][1], parts[1][1])
    w = [(l - top).exp()[..., None] for _, l in parts]
    joined = sum(o.float() * x for (o, _), x in zip(parts, w)) / sum(w)
    keys = [[paged.read(x.np_pages, x.pt[0, i // 16], i % 16, h, 64, x.kg, x.vg) for i in range(x.lengths[0])] for x in (a, b) for h in (0, 1)]
    for g in range(8):
        h = g // 4
        K, V = (np.array([kv[i] for kv in keys[h] + keys[2 + h]]) for i in (0, 1))
        z = K @ f32(q)[0, g].astype(np.float64) / 8
        al = np.exp(z - z.max())
        want = (al / al.sum()) @ V
        assert np.all(np.abs(f32(joined)[0, g] - want) <= 2.0 ** -8 * np.abs(V).max())


def test_calls_on_two_streams_at_once():
    p = Pool("int4", [3000, 2000], [1, 1], d=128, page=16).fill()
    q = [queries(p, 8, seed=s) for s in (1, 2)]
    want = [p.cache.attend(x, p.cu_t) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in q]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(p.cache.attend(q[i], p.cu_t))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_binding_refuses():
    p = Pool("int4", [20], [1]).fill()
    q = queries(p, 2)
    k = torch.randn(1, 2, 64, device="cuda").to(BF16)
    rot = tkv.Rotary(tkv.rope_table(32, 64), [0] * 16 + [1] * 16)
    pos = ints([[1], [2]])
    bad = [lambda: p.cache.attend(q.float(), p.cu_t), lambda: p.cache.attend(q[:, :3], p.cu_t), lambda: p.cache.attend(q, p.cu_t.long()),
           lambda: p.cache.attend(q, p.cu_t[:1]), lambda: p.cache.attend(q.cpu(), p.cu_t), lambda: p.cache.attend(q, p.cu_t, window=-1),
           lambda: p.cache.attend(q, p.cu_t, scale=float("nan")), lambda: p.cache.attend(q, p.cu_t, out=q[:, :2]),
           lambda: p.cache.append(k, k[:0], p.cu_t), lambda: p.cache.append(k, k.half(), p.cu_t), lambda: p.cache.append(k, k, p.cu_t, positions=pos),
           lambda: p.cache.append(k, k, p.cu_t, rotary=rot), lambda: p.cache.append(k, k, p.cu_t, rotary=rot, positions=pos[:1]),
           lambda: p.cache.append(k, k, p.cu_t, rotary=tkv.Rotary(tkv.rope_table(8, 128)), positions=pos[0]),
           lambda: p.cache.append(k[..., 4:], k[..., 4:], p.cu_t), lambda: p.cache.gather(p.cu_t, 1, dtype=torch.int8),
           lambda: tkv.rope(q, rot, None), lambda: tkv.rope(q.long(), rot, pos), lambda: tkv.rope(q, rot, ints([1])),
           lambda: tkv.rope(q.transpose(1, 2), rot, pos), lambda: tkv.Rotary(rot.table, [0] * 31), lambda: tkv.Rotary(rot.table, [4] * 32),
           lambda: tkv.PagedCache(p.pages, p.table, p.lens.long()), lambda: tkv.PagedCache(p.pages[..., :100], p.table, p.lens),
           lambda: tkv.PagedCache(p.pages.to(BF16), p.table, p.lens), lambda: tkv.PagedCache(p.pages, p.table, p.lens[:0]),
           lambda: tkv.PagedCache(torch.zeros(2, 2, 2, 24, 64, device="cuda", dtype=BF16), p.table, p.lens)]
    for call in bad:
        with pytest.raises(tkv.TkvError) as e:
            call()
        assert e.value.status == tkv.TKV_EINVAL
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    assert tkv.tkv_paged_attention(p.cache._c, q, q.clone(), None, tkv.TKV_BF16, 1, 4, (256, 64), (256, 64), p.cu_t, 1, 20, 0, 0.1,
                                   small, 16) == tkv.TKV_ECAPACITY
    assert p.cache.attend(q[:0], p.cu_t).shape == (0, 4, 64)


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("window,n", [(700, 1), (513, 3), (1500, 2)])
def test_windows_over_items_that_are_cut(kind, dtype, window, n):
    p = Pool(kind, [2900, 31, 760, 1024], [n, n, n, n], d=128, page=32).fill()
    q = queries(p, 4, dtype=dtype)
    want = p.oracle(q, window=window)
    for ln in (2900, 20):
        close(p, *p.cache.attend(q, p.cu_t, max_new=n, max_len=ln, window=window, return_lse=True), want, dtype)


def test_offsets_that_descend_are_reported():
    """Rows that several sequences count: 40 of 65,536 rows each are more tiles than 32 bits count."""
    batch, rows, page, pages_a_seq = 80, 65536, 256, 64
    table, lens = torch.zeros(batch, pages_a_seq, dtype=torch.int32, device="cuda"), ints([page * pages_a_seq] * batch)
    cache = tkv.PagedCache.empty(1, table, lens, num_kv_heads=8, head_dim=64, page_size=page)
    q = torch.zeros(rows, 64, 64, dtype=BF16, device="cuda")
    out = torch.full_like(q, 3.0)
    status = ints([0])
    cache.attend(q, ints([0, rows] * (batch // 2) + [0]), max_new=rows, out=out, status=status)
    assert status.item() == tkv.TKV_EINVAL and bool((out == 3.0).all())
    # one sequence that leaves the rows: it is left out, the others are not
    p = Pool("int4", [100, 60, 40], [1, 1, 1], page=16).fill()
    q = queries(p, 4)
    out = torch.full_like(q, 3.0)
    status.zero_()
    p.cache.attend(q, ints([0, 1, 2, 9]), out=out, status=status)
    assert status.item() == tkv.TKV_EINVAL and bool((out[2] == 3.0).all())
    close(p, out[:2], None, tuple(x[:2] for x in p.oracle(q)), BF16)


@pytest.mark.parametrize("max_len", [64, 2000])
def test_kernels_behind_other_work(max_len):
    """Behind a fill, a copy and an event of another stream, eagerly and captured, each call sees what they wrote."""
    p = Pool("int4", [64, 37, 50], [1, 1, 1], page=16, max_pages=128).fill()
    rot = tkv.Rotary(tkv.rope_table(2048, p.d))
    k, v = (torch.randn(3, p.hkv, p.d, device="cuda").to(BF16) for _ in range(2))
    q0, lens0 = queries(p, 4), p.lens.clone()
    q, out = torch.empty_like(q0), torch.empty_like(q0)
    side, main = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        p.lens.zero_()
        out.fill_(7.0)
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            p.lens.copy_(lens0)
            turned = tkv.rope(q0, rot, lens0)
        p.cache.gather(p.cu_t, 3, lengths=lens0)
        here.wait_stream(side)
        p.cache.append(k, v, p.cu_t, rotary=rot)
        q.copy_(turned)
        p.cache.attend(q, p.cu_t, max_len=max_len, out=out)
        q.zero_()
        p.lens.zero_()

    with torch.cuda.stream(main):
        step()
    torch.cuda.synchronize()
    p.lens.copy_(lens0)
    want = p.cache.attend(tkv.rope(q0, rot, lens0), p.cu_t, max_len=max_len)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(5):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)


def test_threads_and_graphs_side_by_side():
    """Four threads, two of them on one stream, rotate and attend beside a graph that is replayed on a fifth stream."""
    import threading
    p = Pool("int4", [3000, 2000], [1, 1], d=128, page=16).fill()
    rot, pos = tkv.Rotary(tkv.rope_table(4096, 128)), [ints([i, 3000 - i]) for i in range(5)]
    q = [queries(p, 4, seed=s) for s in range(5)]
    want = [p.cache.attend(tkv.rope(q[i], rot, pos[i], inverse=i % 2), p.cu_t) for i in range(5)]
    shared, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    streams = [shared, shared, torch.cuda.Stream(), torch.cuda.Stream()]
    with torch.cuda.graph(graph, stream=shared):
        replayed = p.cache.attend(tkv.rope(q[4], rot, pos[4]), p.cu_t)
    torch.cuda.synchronize()
    got, failed = [[] for _ in range(4)], []

    def run(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(40):
                    got[i].append(p.cache.attend(tkv.rope(q[i], rot, pos[i], inverse=i % 2), p.cu_t))
        except Exception as e:   # noqa: BLE001 -- shown below
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    replays = []
    with torch.cuda.stream(torch.cuda.Stream()):
        for _ in range(40):
            graph.replay()
            replays.append(replayed.clone())
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    assert all(torch.equal(x, want[i]) for i in range(4) for x in got[i]) and all(torch.equal(x, want[4]) for x in replays)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d,pairs,interleaved", [(64, 32, False), (64, 32, True), (76, 38, False), (76, 34, True), (74, 37, False), (70, 20, True),
                                                (600, 4, False), (600, 4, True)])
def test_rope_pieces_of_every_size(dtype, d, pairs, interleaved):
    """Rows that start 0 .. 8 elements behind a 16-byte boundary, into rows that start elsewhere: the same bits, the rest as it was."""
    rows, heads = 13, 5
    rot = tkv.Rotary(tkv.rope_table(100, 2 * pairs), [j % 3 for j in range(pairs)], interleaved)
    pos = torch.randint(0, 100, (3, rows), device="cuda", dtype=torch.int32)
    base = torch.randn(rows, heads, d + 16, device="cuda").to(dtype)
    for shift, to in ((0, 0), (8, 0), (4, 4), (2, 4), (1, 0), (0, 3), (6, 2)):
        x = base[:, :, shift:shift + d]
        into = torch.full((rows, heads, d + 24), 7.0, device="cuda", dtype=dtype)
        y = into[:, :, to:to + d]
        tkv.rope(x, rot, pos, out=y)
        check_rotation(y, x, rot.table, pos.cpu().numpy(), [j % 3 for j in range(pairs)], interleaved, False)
        assert torch.equal(y, tkv.rope(x.contiguous(), rot, pos)) and (into[:, :, :to] == 7).all() and (into[:, :, to + d:] == 7).all()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths,n,G,page,window", [
    ([3000], [6], 5, 16, 0), ([700, 0, 33, 1290, 20], [6, 2, 33, 0, 20], 3, 32, 0), ([300, 2100], [40, 3], 8, 16, 0),
    ([1200, 90], [9, 9], 2, 64, 100), ([520, 3], [30, 5], 1, 16, 1), ([64], [64], 4, 16, 0)])
def test_tiles_of_32_rows(dtype, d, lengths, n, G, page, window):
    """What the host expects to be long (the hint says so) is taken 32 rows at a time; the same steps said to be short are not."""
    p = Pool("int4", lengths, n, d=d, page=page).fill()
    q = queries(p, G, dtype=dtype)
    want = p.oracle(q, window=window)
    for ln in (1 << 30, 1):
        out = torch.full((q.shape[0] + 2, q.shape[1], d), 5.0, device="cuda", dtype=dtype)
        padded = torch.cat([q, q[:1], q[:1]])
        _, lse = p.cache.attend(padded, p.cu_t, max_new=max(n), max_len=ln, window=(1 << 30 if window == 0 else window), out=out, return_lse=True)
        close(p, out[:-2], lse[:-2], want, dtype)
        assert (out[-2:] == 5.0).all()


def test_bad_values_in_tiles_of_32_rows():
    """A NaN, an infinity and a bad page where only some of 32 rows look."""
    p = Pool("int4", [400, 130], [10, 7], page=16).fill()
    k, v = (torch.randn(4, 2, 64, device="cuda") for _ in range(2))
    v[0, 0, 3], v[1, 1, 9], k[2, 0, 1], v[3, 0, 40] = float("nan"), float("inf"), float("nan"), -float("inf")
    p.cache.append(k.to(BF16), v.to(BF16), ints([0, 2, 4]))        # the last two positions of both
    p.sync_back()
    p.pt[0, 3] = p.num_pages + 5
    p.table.copy_(torch.tensor(p.pt))
    q = queries(p, 4)
    status = ints([0])
    out = f32(p.cache.attend(q, p.cu_t, max_new=10, max_len=1 << 30, status=status))
    assert status.item() == tkv.TKV_ECAPACITY
    with np.errstate(all="ignore"):
        want = p.oracle(q)[0]
    some = np.isfinite(want)
    assert np.array_equal(np.isfinite(out), some) and some.any() and not some.all()
    # p's rounding 2^-11 and the sums' 2^-14 of at most max |V| < 6, the result's 2^-8: below 2^-7 (1 + |o|)
    assert np.all(np.abs(out[some] - want[some]) <= 2.0 ** -7 * (1 + np.abs(want[some])))
