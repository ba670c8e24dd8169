"""The oracle of 8-bit pages and of beam search, against library routines, closed forms and hand-worked cases; refusals without a GPU."""
import ctypes

import numpy as np
import pytest
import torch

import tiered_kv_cache_gqa_gb300 as tkv
from oracle import beam, fp8, paged8
from test_oracle_paged import cache, call_append


@pytest.mark.parametrize("d", [64, 128])
def test_every_byte_of_a_record_has_one_place(d):
    p, c = np.arange(16)[:, None], np.arange(d)
    both = np.concatenate([paged8.k_place(p, c, d).reshape(-1), paged8.v_place(p, c, d).reshape(-1)])
    assert np.array_equal(np.sort(both), np.arange(32 * d))
    # by hand: K's channels come 64 at a time, V's positions in pairs
    assert paged8.k_place(3, 5, d) == 3 * 64 + 5 and paged8.v_place(0, 0, d) == 16 * d and paged8.v_place(1, 0, d) == 16 * d + 1
    assert paged8.v_place(2, 0, d) == 16 * d + 16 and paged8.v_place(0, 1, d) == 16 * d + 2 and paged8.v_place(8, 0, d) == 24 * d
    assert d == 64 or paged8.k_place(3, 69, d) == 1024 + 3 * 64 + 5


@pytest.mark.parametrize("amax,e", [(448.0, 0), (449.0, 1), (224.0, -1), (225.0, 0), (0.0, -32), (1.75, -8), (1.76, -7), (3.5, -7), (1e-30, -32), (1e38, 31),
                                    (448.0 * 2.0 ** 31, 31), (448.0 * 2.0 ** -32, -32), (np.nextafter(np.float32(448), np.float32(500)), 1)])
def test_exponents_by_hand(amax, e):
    assert paged8.exponent(amax) == e


def test_codes_against_the_library():
    rng = np.random.default_rng(0)
    for e in (-32, -9, 0, 7, 31):
        x = (rng.standard_normal(5000) * 100 * 2.0 ** e).astype(np.float32)
        x[:4] = [0.0, -0.0, 448.0 * 2.0 ** e, -1000.0 * 2.0 ** e]
        want = (torch.tensor(x).double() * 2.0 ** -e).clamp(-448, 448).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(paged8.encode(x, e), want)
    assert list(paged8.encode(np.array([np.inf, -np.inf, np.nan], np.float32), 3)) == [0x7F] * 3


def test_a_block_that_fills_up_row_by_row():
    """The exponent never falls, what was there keeps its value but for subnormals of the new scale, and a new block begins anew."""
    d, rng = 64, np.random.default_rng(1)
    rec = rng.integers(0, 256, paged8.record_bytes(d)).astype(np.uint8)
    sizes = [1.0, 0.1, 500.0, 3.0, 1e6]
    x = [(rng.standard_normal((2, d)) * s).astype(np.float32) for s in sizes]
    es, before = [], None
    for i in range(len(sizes)):
        paged8.append_block(rec, i, x[i][:1], x[i][1:])
        es.append(paged8.exponents(rec, d))
        K, V = paged8.rows(rec, d)
        for which, y in enumerate((K, V)):
            step = 2.0 ** (es[i][which] - 9)                        # the format's smallest step
            assert np.all(np.abs(y[i] - x[i][which]) <= np.maximum(2.0 ** -4 * np.abs(x[i][which]), step / 2))
            if before is not None:
                far = np.abs(before[which][:i]) >= 2.0 ** (es[i][which] - 6)
                assert np.array_equal(y[:i][far], before[which][:i][far])
                assert np.all(np.abs(y[:i] - before[which][:i]) <= step / 2)
        before = (K, V)
    assert es == sorted(es) and es[0] < es[2] < es[4]
    paged8.append_block(rec, 0, x[1][:1], x[1][1:])
    assert paged8.exponents(rec, d) == tuple(paged8.exponent(np.abs(y).max()) for y in x[1])
    # all at once, what no later row makes larger: the same bytes as row by row
    one, each = (np.zeros(paged8.record_bytes(d), np.uint8) for _ in range(2))
    k, v = (np.sort(rng.standard_normal((16, d)).astype(np.float32), axis=0)[::-1] for _ in range(2))
    k[0], v[0] = 5.0, 5.0
    paged8.append_block(one, 0, k, v)
    for i in range(16):
        paged8.append_block(each, i, k[i:i + 1], v[i:i + 1])
    assert np.array_equal(one, each)


def test_attention_against_the_library():
    rng = np.random.default_rng(2)
    d, hkv, page, lengths, n = 64, 2, 16, [37, 0, 5], [3, 0, 1]
    pages = np.zeros((8, hkv, 1, paged8.record_bytes(d)), np.uint8)
    table = np.array([[5, 0, 3], [0, 0, 0], [7, 0, 0]], np.int32)
    k, v = (rng.standard_normal((42, hkv, d)).astype(np.float32) for _ in range(2))
    paged8.append(pages, table, lengths, [0, 37, 37, 42], page, k, v)
    q = rng.standard_normal((4, 6, d))
    for window in (0, 7):
        out, lse, _, _, _ = paged8.attend(q, pages, table, lengths, [0, 3, 3, 4], page, window)
        for b, (r0, m) in ((0, (0, 3)), (2, (3, 1))):
            for h in range(6):
                at, K, V, _ = paged8.sequence(pages, table, b, lengths[b], page, h // 3)
                last = np.arange(lengths[b] - m, lengths[b])[:, None]
                mask = torch.tensor((at <= last) & ((at > last - window) if window else True))
                want = torch.nn.functional.scaled_dot_product_attention(*(torch.tensor(x)[None] for x in (q[r0:r0 + m, h], K, V)), attn_mask=mask[None])[0]
                assert np.allclose(out[r0:r0 + m, h], want.numpy(), rtol=1e-12, atol=1e-12)
    assert np.abs(K).max() < 10 and lse.shape == (4, 6)


def test_selection_against_the_library_and_by_hand():
    rng = np.random.default_rng(3)
    x, s = rng.standard_normal((3, 4, 50)) * 3, -rng.random((3, 4)) * 5
    want = (torch.log_softmax(torch.tensor(x), -1) + torch.tensor(s)[..., None]).flatten(1).topk(9)
    best, beams, tokens = beam.select(x, s, 9)
    assert np.allclose(best, want[0].numpy(), rtol=1e-12) and np.array_equal(beams * 50 + tokens, want[1].numpy())
    # all equal: the first places; a finished beam has its own score; a beam without a score and one with a NaN have nothing
    x, s = np.zeros((1, 3, 4)), np.zeros((1, 3))
    assert beam.select(x, s, 5)[2].tolist() == [[0, 1, 2, 3, 0]] and beam.select(x, s, 5)[1].tolist() == [[0, 0, 0, 0, 1]]
    best, beams, tokens = beam.select(x, s, 4, np.array([[0, 1, 0]]), 2)
    assert best[0, 0] == 0.0 and beams[0].tolist() == [1, 0, 0, 0] and tokens[0].tolist() == [2, 0, 1, 2]
    s[0, 0], x[0, 1, 3], x[0, 2, :3] = -np.inf, np.nan, -np.inf
    best, beams, tokens = beam.select(x, s, 3)
    assert beams[0].tolist() == [2, -1, -1] and tokens[0].tolist() == [3, -1, -1] and best[0, 0] == 0.0


def test_reordering_by_hand():
    table = np.array([[0, 1, 2], [3, 4, 5], [6, 7, 8]], np.int32)
    pages = np.arange(9 * 16, dtype=np.uint8).reshape(9, 1, 1, 16, 1).repeat(2, 2)
    t, (p,) = beam.reorder(table, [20, 20, 20], np.array([[1, 0, 1]]), 16, [pages])
    assert t.tolist() == [[3, 1, 2], [0, 4, 5], [3, 7, 8]]
    for to, frm in ((1, 4), (4, 1), (7, 4)):                        # the current pages: rows 0 .. 3 come from the parent's
        assert np.array_equal(p[to, :, :, :4], pages[frm, :, :, :4]) and np.array_equal(p[to, :, :, 4:], pages[to, :, :, 4:])
    t, (p,) = beam.reorder(table, [32, 32, 32], np.array([[2, -1, 2]]), 16, [pages])
    assert t.tolist() == [[6, 7, 2], [3, 4, 5], [6, 7, 8]] and np.array_equal(p, pages)
    for lengths, parents in (([20, 21, 20], [[1, 1, 1]]), ([49, 49, 49], [[1, 1, 1]]), ([20] * 3, [[3, 9, -5]])):
        t, (p,) = beam.reorder(table, lengths, np.array(parents), 16, [pages])
        assert np.array_equal(t, table) and np.array_equal(p, pages)


# ------------------------------------------------------------------ refusals without a GPU
def test_calls_on_8_bit_pages_refuse_what_the_others_do():
    c = lambda **kw: cache(kv_type=tkv.TKV_E4M3, **kw)   # noqa: E731
    for kw in (dict(pages=0x10008), dict(head_dim=96), dict(page_size=8), dict(batch=0), dict(max_pages=1 << 27)):
        assert call_append(c(**kw)) == tkv.TKV_EINVAL
    assert call_append(c(), dtype=tkv.TKV_E4M3) == tkv.TKV_EINVAL and call_append(c(), dtype=tkv.TKV_FP32) == tkv.TKV_EINVAL
    assert call_append(c(), rows=0) == tkv.TKV_OK
    assert tkv.tkv_paged_gather(c(), 0x100000, 0x200000, tkv.TKV_E4M3, 4, (128, 64), (128, 64), 0x300000, stream=1) == tkv.TKV_EINVAL
    assert tkv.tkv_paged_attention(c(), 0x100000, 0x200000, None, tkv.TKV_FP32, 4, 4, (256, 64), (256, 64), 0x300000, 1, 64, 0, 0.1, 0x400000, 1 << 40,
                                   stream=1) == tkv.TKV_EINVAL


def select(**kw):
    a = dict(logits=0x100000, dtype=tkv.TKV_BF16, batch=2, beams=3, vocab=100, strides=(300, 100), scores=0x200000, finished=None, eos=0, count=3,
             out_scores=0x300000, out_beams=0x400000, out_tokens=0x500000, workspace=0x600000, workspace_bytes=1 << 40)
    a.update(kw)
    return tkv.tkv_beam_select(*a.values(), stream=1)


@pytest.mark.parametrize("kw", [
    dict(logits=0), dict(logits=0x100001), dict(dtype=tkv.TKV_INT4), dict(dtype=tkv.TKV_E4M3), dict(batch=-1), dict(beams=0), dict(beams=65), dict(vocab=0),
    dict(vocab=1 << 30), dict(strides=(-300, 100)), dict(strides=(300, -1)), dict(scores=0), dict(scores=0x200002), dict(finished=0x700000, eos=100),
    dict(finished=0x700000, eos=-1), dict(count=0), dict(count=65), dict(out_scores=0), dict(out_beams=0), dict(out_tokens=0x500001), dict(workspace=0x600008),
    dict(batch=1 << 40)])
def test_selection_refuses(kw):
    assert select(**kw) == tkv.TKV_EINVAL


def test_an_empty_selection_does_nothing():
    assert select(batch=0) == tkv.TKV_OK and tkv.tkv_beam_select_workspace(tkv.TKV_BF16, 0, 3, 100, 3) == 0
    assert tkv.tkv_beam_select_workspace(tkv.TKV_BF16, 2, 65, 100, 3) == 0


def reorder(descs, beams=2, parents=0x700000, num=None, status=None):
    a = (tkv.PagedDesc * len(descs))(*descs)
    return tkv.tkv_paged_reorder(a, len(descs) if num is None else num, parents, beams, status, stream=1)


@pytest.mark.parametrize("call", [
    lambda: reorder([cache(batch=4)], beams=0), lambda: reorder([cache(batch=4)], beams=3), lambda: reorder([cache(batch=66)], beams=33),
    lambda: reorder([cache(batch=4)], parents=0), lambda: reorder([cache(batch=4)], parents=0x700002), lambda: reorder([cache(batch=4)], num=0),
    lambda: reorder([cache(batch=4)], status=0x800001), lambda: reorder([cache(batch=4), cache(batch=2)]), lambda: reorder([cache(batch=4), cache(batch=4, page_table=0x21000)]),
    lambda: reorder([cache(batch=4), cache(batch=4, lengths=0x31000)]), lambda: reorder([cache(batch=4), cache(batch=4, max_pages=5)]),
    lambda: reorder([cache(batch=4), cache(batch=4, page_size=32)]), lambda: reorder([cache(batch=4), cache(batch=4, pages=0)]),
    lambda: reorder([cache(batch=4, page_size=65536, num_kv_heads=1 << 12)])])
def test_reordering_refuses(call):
    assert call() == tkv.TKV_EINVAL


def test_binding_refuses_host_tensors():
    t = torch.zeros(2, 3, 10)
    for call in (lambda: tkv.beam_select(t, t[..., 0]), lambda: tkv.PagedLayers([]), lambda: tkv.PagedLayers([t])):
        with pytest.raises(tkv.TkvError) as e:
            call()
        assert e.value.status == tkv.TKV_EINVAL


def test_status_words_and_enumeration():
    assert (tkv.TKV_INT4, tkv.TKV_E4M3) == (3, 4)
    assert ctypes.sizeof(tkv.PagedDesc) == 72 and fp8.DECODE_TABLE[0x7E] == 448.0
