"""Pins for the oracle of the paged-cache operators, against closed forms and torch's own routines, and the
refusals of the C calls and of the binding that need no GPU."""
import ctypes

import numpy as np
import pytest
import torch

import tiered_kv_cache_gqa_gb300 as tkv
from oracle import fp8, paged

F32 = np.float32


def table(n, pairs):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(pairs) / pairs)
    return np.stack([np.cos(a), np.sin(a)], -1).astype(F32)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(0)
    x, t = rng.standard_normal((5, 3, 20)).astype(F32), table(40, 6)
    pos, axis = rng.integers(0, 40, (2, 5)), [0, 0, 1, 1, 0, 1]
    y = paged.rotate(x, t, pos, axis, interleaved)
    for j in range(6):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + 6)
        w = (x[:, :, a] + 1j * x[:, :, b].astype(np.float64)) * (t[pos[axis[j]], j, 0] + 1j * t[pos[axis[j]], j, 1].astype(np.float64))[:, None]
        # three roundings of values up to |x0| + |x1|
        tol = 3 * 2.0 ** -24 * (np.abs(x[:, :, a]) + np.abs(x[:, :, b]))
        assert np.all(np.abs(y[:, :, a] - w.real) <= tol) and np.all(np.abs(y[:, :, b] - w.imag) <= tol)
    assert np.array_equal(y[:, :, 12:], x[:, :, 12:])
    back = paged.rotate(y, t, pos, axis, interleaved, inverse=True)
    # turned forth and back, each way with three roundings, the table's own rounding (its squares add up to 1 +- 2^-23)
    assert np.max(np.abs(back - x)) <= 8 * 2.0 ** -23 * np.max(np.abs(x)) * 2


def test_records_hold_what_was_put():
    rng = np.random.default_rng(1)
    for d in (64, 128):
        rec = rng.integers(0, 256, 18 * d).astype(np.uint8)
        want = {}
        for r in rng.permutation(16):
            for which in (0, 1):
                x = rng.standard_normal(d).astype(F32) * F32(10.0 ** rng.integers(-2, 3))
                q, b = paged.quantise(x, 0.25)
                paged.put(rec, r, which, q, b, d)
                want[r, which] = q * np.repeat(fp8.DECODE_TABLE[b], 16) * 0.25
                # half a step; or what lies above 7 steps, where the scale was rounded down: by 1/16 of it at most in
                # E4M3's normal range (7/16 of a step, less than half), by 2^-10 below 2^-6 (7 * 2^-10 * gain)
                step = np.repeat(fp8.DECODE_TABLE[b], 16) * 0.25
                assert np.all(np.abs(want[r, which] - x) <= np.maximum(0.5 * step, 7 * 2.0 ** -10 * 0.25) * (1 + 1e-6))
        for (r, which), w in want.items():
            assert np.array_equal(paged.get(rec, r, which, d, 0.25), w)


def test_quantise_special_blocks():
    x = np.zeros(64, F32)
    x[16:32] = 7.0
    x[40], x[50] = np.inf, np.nan
    q, b = paged.quantise(x, 1.0)
    assert not q[:16].any() and b[0] == 0 and np.all(q[16:32] == 7) and fp8.DECODE_TABLE[b[1]] == 1.0
    assert b[2] == 0x7F and b[3] == 0x7F and not q[32:].any()


def test_attention_is_softmax_attention():
    rng = np.random.default_rng(2)
    hkv, G, d, ps = 2, 3, 64, 16
    pages = rng.standard_normal((5, hkv, 2, ps, d))
    pt, lengths, cu = np.array([[3, 0], [1, 4]]), np.array([20, 5]), np.array([0, 2, 3])
    q = rng.standard_normal((4, hkv * G, d))
    out, lse, *_ = paged.attend(q, pages, pt, lengths, cu, ps, hkv, window=7)
    rows = [(0, 0, 18), (1, 0, 19), (2, 1, 4)]
    for row, b, last in rows:
        at = range(max(0, last - 6), last + 1)
        for h in range(hkv * G):
            K, V = (torch.tensor(np.array([pages[pt[b, p // ps], h // G, i, p % ps] for p in at])) for i in (0, 1))
            o = torch.nn.functional.scaled_dot_product_attention(torch.tensor(q[row, h])[None], K, V)
            assert np.allclose(out[row, h], o[0].numpy(), rtol=0, atol=1e-12)
            assert abs(lse[row, h] - torch.logsumexp(K @ torch.tensor(q[row, h]) / 8, 0).item()) < 1e-12
    assert np.isnan(out[3]).all()
    out, lse, *_ = paged.attend(q, pages, pt, np.array([0, 1]), cu, ps, hkv)
    assert not out[:2].any() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2]).all()


# ------------------------------------------------------------------ refusals without a GPU
def rotary(**kw):
    d = tkv.RotaryDesc()
    d.table, d.positions, d.axis_stride, d.max_positions, d.pairs, d.num_axes = 0x10000, 0x20000, 8, 64, 32, 1
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def cache(**kw):
    c = tkv.PagedDesc()
    c.pages, c.page_table, c.lengths, c.num_pages, c.kv_type = 0x10000, 0x20000, 0x30000, 8, tkv.TKV_INT4
    c.num_kv_heads, c.head_dim, c.page_size, c.batch, c.max_pages = 2, 64, 16, 1, 4
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def call_rope(rot=None, x=0x100000, out=0x200000, dtype=tkv.TKV_BF16, rows=8, heads=2, d=64, xs=(128, 64), os=(128, 64)):
    return tkv.tkv_rope(rot or rotary(), x, out, dtype, rows, heads, d, xs, os, stream=1)


@pytest.mark.parametrize("kw", [
    dict(rot=rotary(table=0)), dict(rot=rotary(table=0x10004)), dict(rot=rotary(positions=0)), dict(rot=rotary(pairs=0)),
    dict(rot=rotary(pairs=33)), dict(rot=rotary(pairs=257), d=1024), dict(rot=rotary(num_axes=5)), dict(rot=rotary(num_axes=0)),
    dict(rot=rotary(pair_axis=(ctypes.c_uint8 * 256)(*[1] * 256))), dict(rot=rotary(max_positions=0)), dict(x=0), dict(out=0), dict(x=0x100001),
    dict(dtype=tkv.TKV_INT4), dict(dtype=9), dict(rows=-1), dict(heads=0), dict(os=(64, 64)), dict(os=(0, 64)),
    dict(os=(128, 32)), dict(os=(-128, 64)), dict(xs=(-128, 64)), dict(x=0x200000, xs=(256, 64)),
])
def test_rope_refuses(kw):
    assert call_rope(**kw) == tkv.TKV_EINVAL


def call_append(c=None, rot=None, k=0x100000, v=0x200000, dtype=tkv.TKV_BF16, rows=4, ks=(128, 64), vs=(128, 64), cu=0x300000):
    return tkv.tkv_paged_append(c or cache(), rot, k, v, dtype, rows, ks, vs, cu, stream=1)


CACHES = [dict(pages=0), dict(pages=0x10008), dict(page_table=0), dict(lengths=0), dict(kv_type=tkv.TKV_FP32), dict(kv_type=7),
          dict(head_dim=96), dict(page_size=8), dict(page_size=24), dict(page_size=1 << 17), dict(batch=0), dict(max_pages=0),
          dict(num_pages=0), dict(num_kv_heads=0), dict(max_pages=1 << 27)]


@pytest.mark.parametrize("kw", [dict(c=cache(**x)) for x in CACHES] + [
    dict(dtype=tkv.TKV_FP32), dict(c=cache(kv_type=tkv.TKV_FP16)), dict(k=0), dict(v=0), dict(k=0x100008), dict(ks=(132, 64)),
    dict(vs=(128, 60)), dict(ks=(-128, 64)), dict(rows=-1), dict(rows=1 << 31), dict(cu=0), dict(rot=rotary(table=0)),
    dict(rot=rotary(num_axes=2, positions=0)), dict(rot=rotary(pairs=33)),
])
def test_append_refuses(kw):
    assert call_append(**kw) == tkv.TKV_EINVAL


@pytest.mark.parametrize("kw", [dict(c=cache(**x)) for x in CACHES] + [
    dict(dtype=tkv.TKV_INT4), dict(k=0), dict(k=0x200000), dict(k=0x100008), dict(ks=(64, 64)), dict(ks=(0, 64)), dict(vs=(128, 60)),
    dict(dtype=tkv.TKV_FP32, ks=(130, 64)), dict(rows=-1), dict(cu=0)])
def test_gather_refuses(kw):
    a = dict(c=cache(), k=0x100000, v=0x200000, dtype=tkv.TKV_BF16, rows=4, ks=(128, 64), vs=(128, 64), cu=0x300000)
    a.update(kw)
    assert tkv.tkv_paged_gather(a["c"], a["k"], a["v"], a["dtype"], a["rows"], a["ks"], a["vs"], a["cu"], stream=1) == tkv.TKV_EINVAL


@pytest.mark.parametrize("kw", [dict(c=cache(**x)) for x in CACHES] + [
    dict(hq=3), dict(hq=0), dict(q=0), dict(out=0), dict(q=0x100008), dict(work=0x400008), dict(dtype=tkv.TKV_FP32),
    dict(c=cache(kv_type=tkv.TKV_FP16)), dict(qs=(260, 64)), dict(os=(256, 0)), dict(os=(-256, 64)), dict(new=0), dict(ln=0),
    dict(window=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(rows=-1), dict(rows=0x7FFFFFFF, hq=16), dict(cu=0)])
def test_attention_refuses(kw):
    a = dict(c=cache(), q=0x100000, out=0x200000, dtype=tkv.TKV_BF16, rows=4, hq=4, qs=(256, 64), os=(256, 64), cu=0x300000,
             new=1, ln=64, window=0, scale=0.125, work=0x400000)
    a.update(kw)
    assert tkv.tkv_paged_attention(a["c"], a["q"], a["out"], None, a["dtype"], a["rows"], a["hq"], a["qs"], a["os"], a["cu"],
                                   a["new"], a["ln"], a["window"], a["scale"], a["work"], 1 << 40, stream=1) == tkv.TKV_EINVAL


def test_empty_steps_do_nothing():
    assert call_rope(rows=0) == tkv.TKV_OK and call_append(rows=0) == tkv.TKV_OK
    assert tkv.tkv_paged_attention_workspace(cache(), 3, 1) == 0


def test_binding_refuses_host_tensors():
    t = torch.zeros(4, 2, 2)
    for call in (lambda: tkv.Rotary(t), lambda: tkv.PagedCache(torch.zeros(1, 1, 2, 16, 64, dtype=torch.bfloat16), t, t),
                 lambda: tkv.rope(t, None, None)):
        with pytest.raises(tkv.TkvError) as e:
            call()
        assert e.value.status == tkv.TKV_EINVAL


@pytest.mark.parametrize("cname,pyname", [("tkv_rotary", "RotaryDesc"), ("tkv_paged", "PagedDesc")])
def test_descriptors_match_the_header(cname, pyname):
    from test_abi import header_struct_fields
    assert [f[0] for f in getattr(tkv, pyname)._fields_] == header_struct_fields(cname)


def test_unaligned_and_overlapping_arguments_are_refused():
    """Words that a kernel reads as int32 or fp32 lie on 4 bytes; a score's scale stays finite in powers of two; out is not q."""
    for c in (cache(page_table=0x20002), cache(lengths=0x30001), cache(k_gain=0x40002), cache(v_gain=0x40003)):
        assert call_append(c) == tkv.TKV_EINVAL
    assert call_append(cu=0x300002) == tkv.TKV_EINVAL and call_append(rot=rotary(positions=0x20001)) == tkv.TKV_EINVAL
    assert call_rope(rot=rotary(positions=0x20002)) == tkv.TKV_EINVAL and call_rope(rows=1 << 31) == tkv.TKV_EINVAL

    def attention(out=0x200000, lse=None, cu=0x300000, scale=0.125, status=None):
        return tkv.tkv_paged_attention(cache(), 0x100000, out, lse, tkv.TKV_BF16, 4, 4, (256, 64), (256, 64), cu, 1, 64, 0, scale,
                                       0x400000, 1 << 40, status=status, stream=1)
    for kw in (dict(out=0x100000), dict(lse=0x500002), dict(cu=0x300001), dict(scale=3e38), dict(status=0x600002)):
        assert attention(**kw) == tkv.TKV_EINVAL
