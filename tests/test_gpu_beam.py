"""Beam search: the choice of continuations and the reordering of paged caches against the oracle, and a run of everything together."""
import numpy as np
import pytest
import torch

import tiered_kv_cache_gqa_gb300 as tkv
from oracle import beam, paged, paged8
from test_gpu_paged import BF16, FP16, FP32, close, f32, ints

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


# ------------------------------------------------------------------ selection
def check(x, scores, count, finished=None, eos=None):
    """beam_select against the oracle: the same beams and tokens, and scores as near as derived here.

    A row's sum: its terms carry ex2's 2^-22 and the rounding of their exponents, 2^-24 |x - m| log2 e times a term that falls as 2 to that
    power, below 2^-24; a thread adds 8 terms and one more number a tile of 8,192 values, then come 5 + 8 joins and the chunks: at
    most 8 + V / 8192 + 40 roundings of 2^-24.  That is the logarithm's absolute error; joining the parts of a total rounds below 2^-40 of
    them, the result to half a step."""
    got = tkv.beam_select(x, scores, count=count, finished=finished, eos=eos)
    s = f32(scores)
    want = beam.select(f32(x), s, count, None if finished is None else finished.cpu().numpy(), eos)
    best, beams, tokens = (t.cpu().numpy() for t in got)
    assert got[0].dtype == FP32 and got[1].dtype == torch.int32 and got[2].dtype == torch.int32 and best.shape == (x.shape[0], count)
    assert np.array_equal(beams, want[1]) and np.array_equal(tokens, want[2])
    some = want[0] > -np.inf
    assert np.array_equal(np.isneginf(best), ~some)
    tol = 2.0 ** -22 + (48 + x.shape[2] / 8192) * 2.0 ** -24 + 2.0 ** -24 * np.abs(want[0][some])
    with np.errstate(over="ignore"):
        assert np.all(np.abs(best[some] - want[0][some].astype(np.float64)) <= tol)
    return got


def logits(shape, dtype, seed=0, scale=2.5):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def scores_of(batch, beams, seed=0):
    g = torch.Generator("cuda").manual_seed(seed + 100)
    return -(torch.rand(batch, beams, generator=g, device="cuda") * 10)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("batch,beams,vocab,count", [(1, 1, 1, 1), (1, 1, 7, 1), (2, 3, 5, 16), (1, 4, 32000, 8), (3, 5, 100003, 5), (2, 64, 1000, 64),
                                                   (1, 64, 70001, 64), (70, 2, 2049, 4), (9, 16, 8193, 32), (1, 1, 262144, 64), (5, 7, 4097, 1)])
def test_selection(dtype, batch, beams, vocab, count):
    check(logits((batch, beams, vocab), dtype, vocab), scores_of(batch, beams), count)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("vocab", [9, 1003, 40000])
def test_values_that_are_equal_or_at_the_ends(dtype, vocab):
    """Ties go to the lowest beam and token; masks of the lowest value, infinities and NaN; rows that a mask leaves empty."""
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    flat, s = torch.zeros(2, 4, vocab, device="cuda", dtype=dtype), torch.zeros(2, 4, device="cuda")
    check(flat, s, min(64, 4 * vocab))
    signs = flat.clone()
    signs[..., ::2] = -0.0
    check(signs, s, 8)
    for x in (low, high, -INF):
        check(torch.full_like(flat, x), s, 9)
    y = logits((3, 4, vocab), dtype, 1)
    y[:, :, vocab // 2:], y[1], y[2, 1] = low, low, -INF
    y[0, 0, 0], y[0, 2, -1], y[2, 3, 1] = NAN, INF, high
    check(y, torch.zeros(3, 4, device="cuda"), 9)
    same = logits((2, 1, vocab), dtype, 2).expand(2, 4, vocab)                 # equal beams: the first, whatever their alignment
    check(same, s, 13)
    check(same.contiguous(), s, 13)
    quantised = (logits((2, 4, vocab), dtype, 3).float()).round().to(dtype)     # many equal values
    check(quantised, s, 32)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("vocab,count", [(50001, 64), (131072, 16), (8192, 3), (300000, 64)])
def test_orders_that_overflow_a_list(dtype, vocab, count):
    """Rising and falling values, a plateau and a saw: every tile brings more than the last."""
    up = torch.linspace(-20, 20, vocab, device="cuda")
    rows = torch.stack([up, up.flip(0), up.clamp(max=0.0), up.abs(), torch.where(up > 19.0, up, 0.0), torch.arange(vocab, device="cuda") % 97 - 50.0])
    check(rows[None].to(dtype).contiguous(), torch.linspace(0, -3, 6, device="cuda")[None].contiguous(), count)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_strides_alignments_and_broadcast(dtype):
    wide = logits((5, 9, 4111), dtype, 5)
    s = scores_of(3, 4)
    for shift in range(9):                                                    # rows that begin anywhere in 16 bytes
        check(wide[:3, :4, shift:shift + 4090], s, 8)
    check(wide[1::2, ::2, 3:4100][:, :4], s[:2].contiguous(), 8)
    check(wide[0:1, :4].expand(3, 4, 4111), s, 8)
    check(wide.transpose(0, 1)[:3, :4], s, 8)
    first = check(wide[:3, :4, 1:4091], s, 8)                                   # the same rows elsewhere in memory: the same bits
    for shift in (0, 2, 7):
        moved = torch.empty(3, 4, 4100, device="cuda", dtype=dtype)[..., shift:shift + 4090]
        moved.copy_(wide[:3, :4, 1:4091])
        again = tkv.beam_select(moved, s, count=8)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_long_rows_that_begin_anywhere(dtype):
    """Chunks of several tiles of rows of every alignment; the same bits where all rows begin on 16 bytes."""
    x, s = logits((20, 8, 70009), dtype, 6)[..., 3:70004], scores_of(20, 8)
    first = check(x, s, 4)
    straight = torch.empty(20, 8, 70016, device="cuda", dtype=dtype)[..., :70001]
    straight.copy_(x)
    assert all(torch.equal(a, b) for a, b in zip(first, tkv.beam_select(straight, s, count=4)))


def test_finished_beams_and_beams_that_are_out():
    x, s = logits((4, 6, 5000), BF16, 7), scores_of(4, 6)
    done = torch.zeros(4, 6, dtype=torch.bool, device="cuda")
    done[0, 2], done[1], done[3, ::2] = True, True, True
    for eos in (0, 2, 4999):
        check(x, s, 12, done, eos)
        check(x, s, 12, done.to(torch.uint8) * 255, eos)
    x[0, 2], x[1, 1] = NAN, INF                                               # of a finished beam's logits nothing is read
    check(x, s, 12, done, 2)
    for bad in (-INF, INF, NAN):
        t = s.clone()
        t[0, 1:], t[1, 3], t[2] = bad, bad, bad
        best, beams, tokens = check(x, t, 12, done, 2)
        assert (beams[2] == -1).all() and (tokens[2] == -1).all() and best[2].isneginf().all()
    first = torch.full((4, 6), -INF, device="cuda")                            # the first step: one beam of each sequence is alive
    first[:, 0] = 0.0
    check(logits((4, 6, 5000), BF16, 8), first, 6)


def test_selection_captured_beside_another_and_on_another_stream():
    x = [logits((2, 4, 30000), BF16, i) for i in range(3)]
    s = [scores_of(2, 4, i) for i in range(3)]
    want = [check(a, b, 8) for a, b in zip(x, s)]
    xin, sin = [torch.empty_like(x[0]) for _ in range(2)], [torch.empty_like(s[0]) for _ in range(2)]
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(tkv.beam_select(xin[i], sin[i], count=8))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for t in range(12):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                xin[i].copy_(x[(t + i) % 3])
                sin[i].copy_(s[(t + i) % 3])
                graphs[i].replay()
                got.append(((t + i) % 3, [o.clone() for o in outs[i]]))
        with torch.cuda.stream(streams[2]):
            got.append((t % 3, tkv.beam_select(x[t % 3], s[t % 3], count=8)))
    torch.cuda.synchronize()
    for i, o in got:
        assert all(torch.equal(a, b) for a, b in zip(o, want[i]))


def test_selection_shares_the_workspace_of_an_attention():
    """Calls of both, one after the other on a stream, without a pause."""
    lens = ints([3000, 500])
    table = torch.arange(2 * 94, dtype=torch.int32, device="cuda").view(2, 94)
    cache = tkv.PagedCache.empty(188, table, lens, num_kv_heads=2, head_dim=64, page_size=32, dtype="e4m3")
    kv = torch.randn(3500, 2, 64, device="cuda").to(BF16)
    cache.append(kv, kv, ints([0, 3000, 3500]))
    q, x, s = torch.randn(2, 8, 64, device="cuda").to(BF16), logits((2, 4, 50000), FP32), scores_of(2, 4)
    a, b = cache.attend(q, ints([0, 1, 2])), tkv.beam_select(x, s)
    for _ in range(30):
        c = cache.attend(q, ints([0, 1, 2]))
        d = tkv.beam_select(x, s)
        assert torch.equal(a, c) and all(torch.equal(i, j) for i, j in zip(b, d))


def test_selection_refuses():
    x, s = logits((2, 3, 100), BF16), scores_of(2, 3)
    done = torch.zeros(2, 3, dtype=torch.bool, device="cuda")
    for call in (lambda: tkv.beam_select(x.long(), s), lambda: tkv.beam_select(x[0], s), lambda: tkv.beam_select(x, s.double()), lambda: tkv.beam_select(x, s.t()),
                 lambda: tkv.beam_select(x, s[:1]), lambda: tkv.beam_select(x, s, count=0), lambda: tkv.beam_select(x, s, count=65),
                 lambda: tkv.beam_select(x.transpose(1, 2), s), lambda: tkv.beam_select(x, s, finished=done), lambda: tkv.beam_select(x, s, finished=done, eos=100),
                 lambda: tkv.beam_select(x, s, finished=done.float(), eos=1), lambda: tkv.beam_select(x, s, finished=done[:1], eos=1),
                 lambda: tkv.beam_select(x, s.cpu()), lambda: tkv.beam_select(x[:, :, :0], s), lambda: tkv.beam_select(x.expand(2, 3, 100), s, finished=done.cpu(), eos=1)):
        with pytest.raises(tkv.TkvError) as e:
            call()
        assert e.value.status == tkv.TKV_EINVAL
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    o = [torch.empty(2, 3, device="cuda", dtype=t) for t in (FP32, torch.int32, torch.int32)]
    assert tkv.tkv_beam_select(x, tkv.TKV_BF16, 2, 3, 100, (300, 100), s, None, 0, 3, *o, small, 16) == tkv.TKV_ECAPACITY
    assert tkv.beam_select(x[:0], s[:0])[0].shape == (0, 3)


# ------------------------------------------------------------------ reordering
SHAPES = {"e4m3": lambda n, h, page, d: (n, h, page // 16, 32 * d + 16), "int4": lambda n, h, page, d: (n, h, page // 16, 18 * d),
          "bf16": lambda n, h, page, d: (n, h, 2, page, d), "fp16": lambda n, h, page, d: (n, h, 2, page, d)}


class Beams:
    """Caches of several layers for groups of beams, on both sides; pages of whole prompts are shared."""

    def __init__(self, groups, beams, length, page=16, kinds=("e4m3",), heads=2, d=64, shared=1, seed=0):
        rng = np.random.default_rng(seed)
        self.groups, self.beams, self.page = groups, beams, page
        columns = -(-(length + 1) // page) + 1
        shared = min(shared, length // page)
        own = groups * beams * (columns - shared)
        self.num_pages = own + groups * shared + 1
        order = rng.permutation(self.num_pages).astype(np.int32)
        self.pt = order[:own].reshape(groups * beams, columns - shared)
        prompt = order[own:own + groups * shared].reshape(groups, shared)
        self.pt = np.concatenate([np.repeat(prompt, beams, axis=0), self.pt], axis=1)
        self.lengths = np.full(groups * beams, length, np.int32)
        self.np_pages, self.pages = [], []
        for kind in kinds:
            shape = SHAPES[kind](self.num_pages, heads, page, d)
            if kind in ("e4m3", "int4"):
                x = rng.integers(0, 256, shape).astype(np.uint8)
                t = torch.tensor(x).cuda()
            else:
                x = rng.integers(-100, 100, shape).astype(np.float32)
                t = torch.tensor(x).cuda().to({"bf16": BF16, "fp16": FP16}[kind])
            self.np_pages.append(x)
            self.pages.append(t)
        self.table, self.lens = ints(self.pt), ints(self.lengths)
        self.caches = [tkv.PagedCache(t, self.table, self.lens) for t in self.pages]
        self.layers = tkv.PagedLayers(self.caches)

    def check(self, parents, status=0):
        word = ints([0])
        self.layers.reorder(ints(parents), status=word)
        self.pt, self.np_pages = beam.reorder(self.pt, self.lengths, np.array(parents), self.page, self.np_pages)
        assert word.item() == status
        assert np.array_equal(self.table.cpu().numpy(), self.pt)
        for t, x in zip(self.pages, self.np_pages):
            assert np.array_equal(t.float().cpu().numpy() if t.dtype != torch.uint8 else t.cpu().numpy(), x)


@pytest.mark.parametrize("kinds", [("e4m3",), ("int4", "bf16"), ("fp16", "e4m3", "int4", "bf16")])
@pytest.mark.parametrize("groups,beams,length,page", [(1, 2, 1, 16), (2, 4, 75, 16), (3, 5, 64, 16), (1, 8, 100, 32), (2, 16, 40, 128), (1, 32, 33, 16),
                                                    (1, 17, 47, 16), (2, 9, 15, 64), (4, 1, 20, 16), (1, 3, 0, 16), (40, 2, 18, 16)])
def test_reordering(kinds, groups, beams, length, page):
    b = Beams(groups, beams, length, page, kinds)
    rng = np.random.default_rng(length)
    b.check(rng.permuted(np.tile(np.arange(beams), (groups, 1)), axis=1))     # a permutation: every beam moves at once
    b.check(rng.integers(0, beams, (groups, beams)))
    b.check(np.zeros((groups, beams), int))                                  # all go on from the first
    b.check(np.tile(np.arange(beams), (groups, 1)))                          # nobody moves
    b.check(rng.integers(-1, beams, (groups, beams)))                        # some keep what they have
    b.check(np.tile(np.arange(beams)[::-1], (groups, 1)))


def test_reordering_of_many_layers_with_heads_of_their_own():
    """More caches than a launch takes, of different types, heads and head sizes; and none of the others is touched."""
    b = Beams(2, 3, 41, 16, ("e4m3",))
    rng = np.random.default_rng(1)
    for i in range(70):
        kind, heads, d = ("e4m3", "int4", "bf16", "fp16")[i % 4], 1 + i % 3, (64, 128)[i % 2]
        x = rng.integers(0, 100, SHAPES[kind](b.num_pages + i % 2, heads, 16, d))
        x = x.astype(np.uint8 if kind in ("e4m3", "int4") else np.float32)
        t = torch.tensor(x).cuda()
        b.np_pages.append(x)
        b.pages.append(t if kind in ("e4m3", "int4") else t.to({"bf16": BF16, "fp16": FP16}[kind]))
        b.caches.append(tkv.PagedCache(b.pages[-1], b.table, b.lens))
    b.layers = tkv.PagedLayers(b.caches)
    for _ in range(3):
        b.check(rng.integers(0, 3, (2, 3)))


def test_a_prompt_that_one_beam_has_is_given_to_the_others():
    b = Beams(1, 4, 44, 16, ("e4m3", "bf16"), shared=0)
    b.check([[2, 2, 2, 2]])
    kk, vv = b.caches[0].gather(ints([0, 44, 88, 132, 176]), 176)
    for i in (0, 1, 3):
        assert torch.equal(kk[44 * i:44 * i + 44].nan_to_num(9.0), kk[88:132].nan_to_num(9.0)) and torch.equal(vv[44 * i:44 * i + 44].nan_to_num(9.0), vv[88:132].nan_to_num(9.0))


def test_reordering_that_makes_no_sense_is_reported():
    b = Beams(3, 3, 41, 16, ("e4m3", "bf16"))
    b.check([[0, 3, 1], [2 ** 31 - 1, 1, 0], [0, 1, 2]], tkv.TKV_EINVAL)         # no such parent: the sequence stays
    b.lengths[4] = 40
    b.lens.copy_(ints(b.lengths))
    b.check([[1, 0, 1], [1, 0, 1], [2, 2, 2]], tkv.TKV_EINVAL)                   # a group whose lengths differ stays
    for far in (16 * b.pt.shape[1] + 1, 2 ** 31 - 1, -1, -2 ** 31):
        b.lengths[3:6] = far
        b.lens.copy_(ints(b.lengths))
        b.check([[0, 0, 1], [1, 0, 1], [1, 2, 2]], tkv.TKV_ECAPACITY)            # lengths outside the table
    b.lengths[3:6] = 16 * b.pt.shape[1]
    b.lens.copy_(ints(b.lengths))
    b.check([[2, 0, 1], [1, 0, 1], [1, 2, 0]])                                   # the table is full: nothing is copied
    b.lengths[:] = 41
    b.lens.copy_(ints(b.lengths))
    b.pt[1, 2], b.pt[8, 2] = -1, b.num_pages
    b.table.copy_(ints(b.pt))
    b.check([[1, 0, 1], [1, 0, 1], [2, 2, 2]], tkv.TKV_ECAPACITY)                # pages that there are not


def test_reordering_of_caches_with_fewer_pages():
    """A beam whose page one cache does not have stays there, and follows in the others."""
    b = Beams(2, 5, 41, 16, ("bf16", "bf16", "e4m3", "fp16"))
    for i, left in ((1, b.num_pages - 7), (2, b.num_pages - 4)):
        b.pages[i], b.np_pages[i] = b.pages[i][:left], b.np_pages[i][:left]
    b.caches = [tkv.PagedCache(t, b.table, b.lens) for t in b.pages]
    b.layers = tkv.PagedLayers(b.caches)
    assert (b.pt[:, 2] >= b.num_pages - 7).any()
    parents = np.array([[1, 2, 3, 4, 0], [4, 0, 0, 1, 1]])
    moved = np.concatenate([np.stack([b.pt[5 * g:5 * g + 5, 2], b.pt[5 * g + parents[g], 2]], 1) for g in range(2)])
    b.check(parents, tkv.TKV_ECAPACITY if (moved >= b.num_pages - 7).any() else 0)
    b.check([[0, 0, 0, 0, 0], [3, 3, 3, 3, 3]], tkv.TKV_ECAPACITY)


def test_reordering_captured_behind_a_selection():
    """Selection, reordering and the next tokens' append in one graph: each replay reads what the last one left."""
    a, b = (Beams(2, 4, 40, 16, ("e4m3", "bf16"), seed=3) for _ in range(2))
    x, s = logits((6, 2, 4, 3001), BF16, 3), scores_of(2, 4)
    kv = torch.randn(6, 2, 8, 2, 64, device="cuda").to(BF16)
    cu = ints(list(range(9)))

    def step(m, xin, sin, k):
        best, beams, tokens = tkv.beam_select(xin, sin)
        m.layers.reorder(beams)
        sin.copy_(best)
        m.lens.add_(1)
        for c in m.caches:
            c.append(k[0], k[1], cu)
        return beams, tokens

    sa, sb = s.clone(), s.clone()
    want = [[t.clone() for t in step(a, x[t], sa, kv[t])] for t in range(6)]
    xin, k = x[0].clone(), kv[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(b, xin, sb, k)
    for t in range(6):
        xin.copy_(x[t])
        k.copy_(kv[t])
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(out, want[t]))
    assert torch.equal(sa, sb) and torch.equal(a.table, b.table) and all(torch.equal(p, q) for p, q in zip(a.pages, b.pages))


def test_reordering_refuses():
    b = Beams(2, 2, 20, 16, ("e4m3", "bf16"))
    other = Beams(2, 2, 20, 16, ("e4m3",))
    for call in (lambda: tkv.PagedLayers([]), lambda: tkv.PagedLayers(b.caches + other.caches), lambda: tkv.PagedLayers([b.caches[0], None]), lambda: tkv.PagedLayers([b.caches[0], b.caches[1], b.caches[0]]),
                 lambda: b.layers.reorder(ints([0, 1, 0, 1])), lambda: b.layers.reorder(ints([[0, 1]])), lambda: b.layers.reorder(ints([[0, 1, 0, 1]]).long()),
                 lambda: b.layers.reorder(ints([[0, 1], [0, 1]]).t()), lambda: b.layers.reorder(ints([[0, 1], [0, 1]]).cpu()), lambda: b.layers.reorder(None),
                 lambda: b.layers.reorder(ints([[0, 1], [0, 1]]), status=torch.zeros(1, device="cuda"))):
        with pytest.raises(tkv.TkvError) as e:
            call()
        assert e.value.status == tkv.TKV_EINVAL
    wide = Beams(1, 32, 20, 16, ("e4m3",))
    wide.check(np.arange(32)[None, ::-1].copy())
    many = tkv.PagedCache(wide.pages[0], torch.zeros(33, 2, dtype=torch.int32, device="cuda"), ints([1] * 33))
    with pytest.raises(tkv.TkvError):
        tkv.PagedLayers([many]).reorder(ints([[0] * 33]))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("kind", ["e4m3", "int4", "bf16"])
def test_beam_search_over_the_caches_of_two_layers(kind):
    """A prompt enters through one beam and is given to the others; then 40 steps of append, attention, selection and reordering.

    The other side keeps a dense copy of every beam's rows as the cache reads them back (each beam's own append into pages that nobody
    shares) and copies whole beams; the pages, read back, and the choices are the same, and the attention is right for them."""
    groups, W, prompt, d, hkv, G, page, vocab, layers, steps = 2, 4, 37, 64, 2, 3, 32, 997, 2, 40
    batch, columns = groups * W, 4
    table = torch.randperm(batch * columns, device="cuda").to(torch.int32).view(batch, columns).contiguous()
    lens = ints([0] * batch)
    dtype = kind if kind in ("e4m3", "int4") else BF16
    caches = [tkv.PagedCache.empty(batch * columns, table, lens, num_kv_heads=hkv, head_dim=d, page_size=page, dtype=dtype) for _ in range(layers)]
    # the other side: the same pages a beam, never shared
    mine = torch.arange(batch * columns, dtype=torch.int32, device="cuda").view(batch, columns)
    other = [tkv.PagedCache.empty(batch * columns, mine, lens, num_kv_heads=hkv, head_dim=d, page_size=page, dtype=dtype) for _ in range(layers)]
    all_layers = tkv.PagedLayers(caches)
    g = torch.Generator("cuda").manual_seed(1)
    rot = tkv.Rotary(tkv.rope_table(256, d))
    rnd = lambda *shape: torch.randn(*shape, generator=g, device="cuda")   # noqa: E731
    words, head = rnd(vocab, 3 * d) * 0.7, rnd(hkv * G * d, vocab) * 0.05

    lens.fill_(prompt)
    k, v = rnd(groups * prompt, hkv, d).to(BF16), rnd(groups * prompt, hkv, d).to(BF16)
    one = ints(np.repeat(np.arange(groups + 1), W)[W - 1:W - 1 + batch + 1] * prompt)      # the first beam of each group has all rows
    cu_all = ints(np.arange(batch + 1) * prompt)
    many = torch.arange(groups, device="cuda").repeat_interleave(W)
    for a, b in zip(caches, other):
        a.append(k, v, one, rotary=rot)
        kk, vv = (x.view(groups, prompt, hkv, d)[many].reshape(-1, hkv, d).contiguous() for x in (k, v))
        b.append(kk, vv, cu_all, rotary=rot)
    all_layers.reorder(torch.zeros(groups, W, dtype=torch.int32, device="cuda"))
    scores = torch.full((groups, W), -INF, device="cuda")
    scores[:, 0] = 0.0
    tokens = torch.zeros(groups, W, dtype=torch.int32, device="cuda")
    cu = ints(np.arange(batch + 1))
    finished = torch.zeros(groups, W, dtype=torch.bool, device="cuda")
    moved = 0
    for step in range(steps):
        lens.add_(1)
        x = words[tokens.clamp(min=0).flatten().long()].view(batch, 3, 1, d)
        n = prompt + step + 1
        hidden = 0.0
        for i, (a, b) in enumerate(zip(caches, other)):
            k, v, q = ((x[:, j] * (1 + 0.1 * i) + torch.arange(h, device="cuda")[None, :, None] * 0.01).to(BF16) for j, h in ((0, hkv), (1, hkv), (2, hkv * G)))
            q = tkv.rope(q, rot, lens - 1)
            a.append(k, v, cu, rotary=rot)
            b.append(k, v, cu, rotary=rot)
            out, lse = a.attend(q, cu, max_len=n, return_lse=True)
            o2, l2 = b.attend(q, cu, max_len=n, return_lse=True)
            assert torch.equal(out, o2) and torch.equal(lse, l2)               # the same rows in other pages
            hidden = hidden + out.float()
        if step % 13 == 0:
            cu_n = ints(np.arange(batch + 1) * n)
            for a, b in zip(caches, other):
                for p, q2 in zip(a.gather(cu_n, batch * n, dtype=FP32), b.gather(cu_n, batch * n, dtype=FP32)):
                    assert torch.equal(p, q2)
            if kind == "e4m3":                                                # and the last layer's attention against 64 bits
                class P:
                    pass
                P.kind, P.d = "e4m3", d
                want = paged8.attend(f32(q).astype(np.float64), caches[-1].pages.cpu().numpy(), table.cpu().numpy(), [n] * batch, np.arange(batch + 1), page)
                close(P, out, lse, want, BF16)
        logit = (hidden.flatten(1) @ head).view(groups, W, vocab).to(BF16)
        want = beam.select(f32(logit), f32(scores), W, finished.cpu().numpy(), 5)
        scores, beams, tokens = tkv.beam_select(logit, scores, finished=finished, eos=5)
        assert np.array_equal(beams.cpu().numpy(), want[1]) and np.array_equal(tokens.cpu().numpy(), want[2])
        finished = finished.gather(1, beams.long()) | (tokens == 5)
        all_layers.reorder(beams)
        moved += int((beams != torch.arange(W, device="cuda")).sum())
        flat = (torch.arange(batch, device="cuda") // W * W + beams.flatten().long())
        for b in other:                                                       # whole beams are copied
            pages = b.pages.view(batch, columns, *b.pages.shape[1:])
            pages.copy_(pages[flat].clone())
        if finished.all():
            finished.zero_()
    assert moved > steps and paged is not None
