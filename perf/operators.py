"""The operators around a paged KV cache: what is measured of them, and their plain forms.

  rope       rotary positions with one or several axes, forward and inverse (its gradient)
  append     rows of k and v into a paged cache, k rotated on the way; 4-bit or 16-bit pages; read back by `gather`
  attention  the queries of a step over a paged cache held in 4 bits, or in 16

The plain forms are elementary torch operations in 32 bits.  A 4-bit page holds, per KV head, groups of 16 positions:
K codes [16][d/2] | K scales [16][d/16] | V codes [16][d/2] | V scales [d/16][16], a code q + 8 in four bits (the even
channel in the low ones), q in -7..7, a scale in E4M3 for 16 channels; the value is q * scale * gain of the head.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
WIDTH = {"bf16": 2.0, "fp16": 2.0, "fp32": 4.0, "int4": 0.5625}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode token's queries, 28 heads: what a launch costs
        dict(name="rope_one_token", op="rope", dtype="bf16", tokens=1, heads=28, head_dim=128, rot_dim=128, axes=1,
             interleaved=False, inverse=False),
        # the query heads of a prompt with text, image and video positions, three axes
        dict(name="rope_video_prompt", op="rope", dtype="bf16", tokens=16384, heads=64, head_dim=128, rot_dim=128, axes=3,
             interleaved=False, inverse=False),
        # the gradient of a partial rotation in 32 bits, adjacent pairs, two axes of an image, odd sizes
        dict(name="rope_gradient_fp32", op="rope", dtype="fp32", tokens=5003, heads=13, head_dim=80, rot_dim=56, axes=2,
             interleaved=True, inverse=True),
        # a decode step: one token a sequence into 4-bit pages
        dict(name="append_decode_int4", op="append", kv="int4", dtype="bf16", batch=8, kv_heads=8, head_dim=128, page=64,
             prior=4096, new=1, axes=1),
        # prompts of several lengths enter the 4-bit cache together
        dict(name="append_prompts_int4", op="append", kv="int4", dtype="bf16", batch=8, kv_heads=8, head_dim=128, page=64,
             prior=301, new=4096, axes=1),
        # prompts with positions on three axes into 16-bit pages
        dict(name="append_prompts_bf16", op="append", kv="bf16", dtype="bf16", batch=5, kv_heads=4, head_dim=128, page=16,
             prior=33, new=2047, axes=3),
        # batch 1, one reasoning chain of 2,512 positions, 28/4 heads
        dict(name="attend_one_chain_int4", op="attention", kv="int4", dtype="bf16", batch=1, q_heads=28, kv_heads=4,
             head_dim=128, page=16, length=2512, ragged=False, new=1, window=0),
        # batch 8, 64/8 heads, 16,384 positions a sequence
        dict(name="attend_batch_int4", op="attention", kv="int4", dtype="bf16", batch=8, q_heads=64, kv_heads=8,
             head_dim=128, page=64, length=16384, ragged=False, new=1, window=0),
        # the largest: a serving batch of mixed lengths up to 65,536, empty and idle sequences among them
        dict(name="attend_serving_int4", op="attention", kv="int4", dtype="bf16", batch=32, q_heads=64, kv_heads=8,
             head_dim=128, page=64, length=65536, ragged=True, new=1, window=0),
        # several drafted tokens a sequence are checked at once
        dict(name="attend_drafts_int4", op="attention", kv="int4", dtype="bf16", batch=4, q_heads=40, kv_heads=8,
             head_dim=128, page=32, length=8192, ragged=True, new=6, window=0),
        # small heads, an odd group, a window, many short sequences
        dict(name="attend_window_d64_int4", op="attention", kv="int4", dtype="fp16", batch=67, q_heads=24, kv_heads=8,
             head_dim=64, page=16, length=1531, ragged=True, new=1, window=700),
        # the same operator over 16-bit pages: 40/8 heads, batch 8, 4,096 positions
        dict(name="attend_batch_bf16", op="attention", kv="bf16", dtype="bf16", batch=8, q_heads=40, kv_heads=8,
             head_dim=128, page=64, length=4096, ragged=False, new=1, window=0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention"])
    if op == "rope":
        tokens, heads = _log(rng, 1, 16384), rng.randint(1, 64)
        head_dim = 2 * rng.randint(8, 128)
        tokens = max(1, min(tokens, 16384 * 64 * 128 // (heads * head_dim * 2)))
        rot_dim = head_dim if rng.random() < 0.6 else 2 * rng.randint(1, head_dim // 2)
        return dict(op="rope", dtype=rng.choice(["bf16", "fp16", "fp32"]), tokens=tokens, heads=heads, head_dim=head_dim,
                    rot_dim=rot_dim, axes=rng.randint(1, 4), interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5)
    head_dim, page, kv_heads = rng.choice([64, 128]), rng.choice([16, 32, 64, 128]), rng.randint(1, 8)
    dtype = rng.choice(["bf16", "fp16"])
    kv = "int4" if rng.random() < 0.7 else dtype
    if op == "append":
        batch = _log(rng, 1, 64)
        new = max(1, min(_log(rng, 1, 4096), 16384 // batch))
        return dict(op="append", kv=kv, dtype=dtype, batch=batch, kv_heads=kv_heads, head_dim=head_dim, page=page,
                    prior=rng.randint(0, 4096), new=new, axes=rng.randint(1, 3))
    batch, group = _log(rng, 1, 128), rng.randint(1, 8)
    most = 7e8 / (batch * kv_heads * head_dim * 2 * WIDTH[kv])
    length = max(1, min(_log(rng, 1, 65536), int(most)))
    new = min(length, rng.choice([1, 1, 1, rng.randint(2, 8)]))
    return dict(op="attention", kv=kv, dtype=dtype, batch=batch, q_heads=group * kv_heads, kv_heads=kv_heads, head_dim=head_dim,
                page=page, length=length, ragged=rng.random() < 0.7, new=new,
                window=rng.choice([0, 0, rng.randint(1, length)]))


def _counts(case):
    """(positions after the step, tokens of the step) of each sequence: a rule of the case alone."""
    b, new = case["batch"], case["new"]
    if case["op"] == "append":   # the first sequence has `new` tokens, the others fewer
        n = [max(1, new * (b - i) // b) for i in range(b)]
        return [(case["prior"] * (i + 1)) // b + n[i] for i in range(b)], n
    if not case["ragged"]:
        return [case["length"]] * b, [new] * b
    lens, n = [], []
    for i in range(b):           # the first is the longest; one in eleven is empty, one in seven idle
        f = 1.0 if i == 0 else (0.02 + 0.98 * ((i * 0.6180339887498949) % 1.0)) ** 2
        lens.append(0 if i % 11 == 7 else max(1, int(case["length"] * f)))
        n.append(0 if i % 7 == 5 else 1 + (new - 1 + 3 * i) % new)
    return lens, n


def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["head_dim"] * WIDTH[case["dtype"]] + case["tokens"] * (case["rot_dim"] * 4 + 4 * case["axes"]),
                "flops": 3 * n * case["rot_dim"]}
    lens, n = _counts(case)
    d, hkv, w = case["head_dim"], case["kv_heads"], WIDTH[case["kv"]]
    if case["op"] == "append":
        t = sum(n)
        rows = t * hkv * d * 2
        return {"bytes": rows * (2 + w) + t * (d * 4 + 4 * case["axes"]) + (rows * (2 + w) if case["kv"] == "int4" else 0),
                "flops": 3 * t * hkv * d}
    w0 = case["window"]
    seen = [0 if not m else l if not w0 else min(l, w0 + m - 1) for l, m in zip(lens, n)]
    pairs = sum(min(max(0, l - m + i + 1), w0 or l) for l, m in zip(lens, n) for i in range(m))
    return {"bytes": sum(seen) * hkv * d * 2 * w + sum(n) * case["q_heads"] * (d * 4 + 4),
            "flops": 4 * case["q_heads"] * d * pairs}


# ------------------------------------------------------------------ inputs
def _table(max_positions, pairs, device):
    freq = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device=device) / pairs)
    angle = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.stack([angle.cos(), angle.sin()], dim=-1).float().contiguous()


def _pair_axis(pairs, axes):
    """Sections of pairs, one an axis, as even as they come."""
    return [min(axes - 1, j * axes // pairs) for j in range(pairs)]


def _positions(g, axes, base, device):
    """Axis 0: `base` (int32, one a token); the others: the rows and columns of images, below 512."""
    more = [torch.randint(0, 512, base.shape, generator=g, device=device, dtype=torch.int32) for _ in range(axes - 1)]
    return torch.stack([base] + more).contiguous()


def _e4m3(x):
    """The nearest E4M3 value (ties to even, saturating at 448) of x >= 0, and its byte."""
    q = x.clamp(max=448.0).to(torch.float8_e4m3fn)
    return q.float(), q.view(torch.uint8)


def _quantise(x, gain):
    """x [..., d] fp32, gain broadcast over [..., 1] -> codes q (-7..7, fp32) [..., d], scale bytes [..., d/16], values."""
    blocks = x.unflatten(-1, (-1, 16))
    amax = blocks.abs().amax(-1)
    scale, byte = _e4m3(amax / (7.0 * gain))
    step = (scale * gain)[..., None]
    q = torch.where(step > 0, (blocks / step).round().clamp(-7, 7), torch.zeros_like(blocks))
    bad = ~torch.isfinite(amax)
    byte = torch.where(bad, torch.full_like(byte, 0x7F), byte)
    q = torch.where(bad[..., None], torch.zeros_like(q), q)
    return q.flatten(-2), byte


def _pack(q):
    c = (q + 8).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _unpack(b):
    return torch.stack([(b & 15).float() - 8, (b >> 4).float() - 8], dim=-1).flatten(-2)


def _record(d):
    """Offsets of a group record: K scales, V codes, V scales, its end."""
    return 8 * d, 9 * d, 17 * d, 18 * d


def _store_int4(k, v, k_gain, v_gain):
    """k, v fp32 [pages, heads, page, d] -> page bytes [pages, heads, page/16, 18 d]."""
    parts = []
    for x, gain in ((k, k_gain), (v, v_gain)):
        q, byte = _quantise(x, gain[:, None, None])
        codes = _pack(q).unflatten(2, (-1, 16)).flatten(3)
        byte = byte.unflatten(2, (-1, 16))
        parts += [codes, (byte if x is k else byte.transpose(-1, -2)).flatten(3)]
    return torch.cat(parts, dim=-1).contiguous()


def _fill(g, case, lens, device):
    """The page pool, the page table and the lengths of a cache whose rows are keys and values as a model makes them:
    normal, one position in a hundred a heavy hitter whose key lies along its head's direction u."""
    b, hkv, d, page = case["batch"], case["kv_heads"], case["head_dim"], case["page"]
    need = [max(1, -(-x // page)) for x in lens]
    total = sum(need) + 2
    order = torch.randperm(total, generator=g, device=device).to(torch.int32)
    table = torch.zeros(b, max(need), dtype=torch.int32)
    at, starts = 0, []
    for n in need:
        starts.append(at)
        at += n
    cols = torch.arange(max(need), device=device)
    first = torch.tensor(starts, device=device)[:, None]
    many = torch.tensor(need, device=device)[:, None]
    table = torch.where(cols < many, order[(first + cols).clamp(max=total - 1)], torch.zeros((), dtype=torch.int32, device=device))
    k_gain = torch.exp2(torch.randint(-9, -6, (hkv,), generator=g, device=device).float()) / 2
    v_gain = torch.exp2(torch.randint(-9, -6, (hkv,), generator=g, device=device).float()) / 2
    u = torch.randn(hkv, d, generator=g, device=device)
    u = u / u.norm(dim=-1, keepdim=True)
    if case["kv"] == "int4":
        pages = torch.empty(total, hkv, page // 16, 18 * d, dtype=torch.uint8, device=device)
    else:
        pages = torch.empty(total, hkv, 2, page, d, dtype=DTYPES[case["kv"]], device=device)
    chunk = max(1, (1 << 26) // (hkv * page * d))
    for p in range(0, total, chunk):
        m = min(chunk, total - p)
        k = torch.randn(m, hkv, page, d, generator=g, device=device)
        hot = torch.rand(m, 1, page, 1, generator=g, device=device) < 0.01
        k += torch.where(hot, 4.0, 0.0) * u[:, None]
        v = torch.randn(m, hkv, page, d, generator=g, device=device)
        if case["kv"] == "int4":
            pages[p:p + m] = _store_int4(k, v, k_gain, v_gain)
        else:
            pages[p:p + m, :, 0] = k.to(pages.dtype)
            pages[p:p + m, :, 1] = v.to(pages.dtype)
    return {"pages": pages, "page_table": table.contiguous(), "lengths": torch.tensor(lens, dtype=torch.int32, device=device),
            "k_gain": k_gain if case["kv"] == "int4" else None, "v_gain": v_gain if case["kv"] == "int4" else None, "u": u}


def prepare(case, seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "rope":
        pairs = case["rot_dim"] // 2
        t = case["tokens"]
        s["x"] = torch.randn(t, case["heads"], case["head_dim"], generator=g, device=device).to(DTYPES[case["dtype"]])
        start = int(torch.randint(0, 16384, (1,), generator=g, device=device))
        s["positions"] = _positions(g, case["axes"], torch.arange(start, start + t, dtype=torch.int32, device=device), device)
        s["table"] = _table(32768, pairs, device)
        s["pair_axis"] = _pair_axis(pairs, case["axes"])
        s["axis_of_pair"] = torch.tensor(s["pair_axis"], device=device)
        return s
    lens, n = _counts(case)
    hkv, d = case["kv_heads"], case["head_dim"]
    s.update(_fill(g, case, lens, device))
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=device)
    s["rows"], s["max_new"], s["max_len"] = cu[-1], max(n), max(lens)
    if case["op"] == "append":
        t = s["rows"]
        s["k"] = torch.randn(t, hkv, d, generator=g, device=device).to(DTYPES[case["dtype"]])
        s["v"] = torch.randn(t, hkv, d, generator=g, device=device).to(DTYPES[case["dtype"]])
        seq, pos = _where(s)
        s["positions"] = _positions(g, case["axes"], pos.to(torch.int32), device)
        s["table"] = _table(16384, d // 2, device)
        s["pair_axis"] = _pair_axis(d // 2, case["axes"])
        s["axis_of_pair"] = torch.tensor(s["pair_axis"], device=device)
        return s
    group = case["q_heads"] // hkv
    q = torch.randn(s["rows"], hkv, group, d, generator=g, device=device) + 0.5 * math.sqrt(d) * s["u"][:, None]
    s["q"] = q.reshape(s["rows"], case["q_heads"], d).to(DTYPES[case["dtype"]])
    return s


# ------------------------------------------------------------------ the framework's operators
def _handles(s):
    """The cache and the rotation that a user's program builds once."""
    import tiered_kv_cache_gqa_gb300 as tkv
    c = s["case"]
    if "rotary" not in s and "table" in s:
        s["rotary"] = tkv.Rotary(s["table"], pair_axis=s["pair_axis"], interleaved=c.get("interleaved", False))
    if "cache" not in s and "pages" in s:
        s["cache"] = tkv.PagedCache(s["pages"], s["page_table"], s["lengths"], k_gain=s["k_gain"], v_gain=s["v_gain"])
    return tkv


def _run_own(s):
    tkv, c = _handles(s), s["case"]
    if c["op"] == "rope":
        return tkv.rope(s["x"], s["rotary"], s["positions"], inverse=c["inverse"])
    if c["op"] == "append":
        s["cache"].append(s["k"], s["v"], s["cu"], rotary=s["rotary"], positions=s["positions"])
        return s["pages"] if c["kv"] != "int4" else s["cache"].gather(s["cu"], s["rows"], dtype=s["k"].dtype)
    return s["cache"].attend(s["q"], s["cu"], max_new=s["max_new"], max_len=s["max_len"], window=c["window"], return_lse=True)


# ------------------------------------------------------------------ the plain forms
def _rotate(x, s, interleaved=False, inverse=False):
    """x fp32 [T, H, d]; the first 2 * pairs channels of a head are rotated."""
    pairs = s["table"].shape[1]
    at = s["positions"].long()[s["axis_of_pair"]].T                                  # [T, pairs]
    cs = s["table"][at, torch.arange(pairs, device=x.device)]                        # [T, pairs, 2]
    c, sn = cs[:, None, :, 0], cs[:, None, :, 1]
    if inverse:
        sn = -sn
    x0, x1 = (x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2]) if interleaved else (x[..., :pairs], x[..., pairs:2 * pairs])
    y0, y1 = x0 * c - x1 * sn, x1 * c + x0 * sn
    y = torch.stack([y0, y1], dim=-1).flatten(-2) if interleaved else torch.cat([y0, y1], dim=-1)
    return torch.cat([y, x[..., 2 * pairs:]], dim=-1)


def _where(s):
    """The sequence and the position of each row of the step."""
    cu, lengths = s["cu"].long(), s["lengths"].long()
    row = torch.arange(s["rows"], device=cu.device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    return seq, lengths[seq] - (cu[seq + 1] - row)


def _plain_append(s):
    c = s["case"]
    page, d = c["page"], c["head_dim"]
    seq, pos = _where(s)
    pg, off = s["page_table"].long()[seq, pos // page], pos % page
    k, v = _rotate(s["k"].float(), s), s["v"].float()
    if c["kv"] != "int4":
        s["pages"][pg, :, 0, off] = k.to(s["pages"].dtype)
        s["pages"][pg, :, 1, off] = v.to(s["pages"].dtype)
        return s["pages"]
    ks, vc, vs, end = _record(d)
    rec = s["pages"].unflatten(2, (page // 16,))
    grp, r = off // 16, off % 16
    kq, kb = _quantise(k, s["k_gain"][:, None])
    vq, vb = _quantise(v, s["v_gain"][:, None])
    parts = [rec[:, :, :, :ks].unflatten(3, (16, d // 2)), rec[:, :, :, ks:vc].unflatten(3, (16, d // 16)),
             rec[:, :, :, vc:vs].unflatten(3, (16, d // 2)), rec[:, :, :, vs:end].unflatten(3, (d // 16, 16)).transpose(3, 4)]
    for part, x in zip(parts, (_pack(kq), kb, _pack(vq), vb)):
        part[pg, :, grp, r] = x
    kq, kb, vq, vb = (part[pg, :, grp, r] for part in parts)                          # read back: [T, H, ...]
    return (_values(kq, kb, s["k_gain"][:, None]).to(s["k"].dtype), _values(vq, vb, s["v_gain"][:, None]).to(s["k"].dtype))


def _values(codes, scales, gain):
    """The fp32 values of codes [..., d/2] with their scale bytes [..., d/16]."""
    return _unpack(codes) * scales.contiguous().view(torch.float8_e4m3fn).float().repeat_interleave(16, dim=-1) * gain


def _read_int4(rec, d, k_gain, v_gain):
    """Group records [..., 18 d] -> K, V fp32 [..., 16, d]."""
    ks, vc, vs, end = _record(d)
    k = _values(rec[..., :ks].unflatten(-1, (16, d // 2)), rec[..., ks:vc].unflatten(-1, (16, d // 16)), k_gain)
    return k, _values(rec[..., vc:vs].unflatten(-1, (16, d // 2)),
                      rec[..., vs:end].unflatten(-1, (d // 16, 16)).transpose(-1, -2), v_gain)


def _plain_attention(s):
    c = s["case"]
    b, hq, hkv, d, page = c["batch"], c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    group, m = hq // hkv, s["max_new"]
    got = s["pages"][s["page_table"].long()]                                         # [B, P, H, ...]
    if c["kv"] == "int4":
        k, v = _read_int4(got, d, s["k_gain"][:, None, None, None], s["v_gain"][:, None, None, None])
        k, v = k.flatten(3, 4), v.flatten(3, 4)
    else:
        k, v = got[:, :, :, 0].float(), got[:, :, :, 1].float()
    del got
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in (k, v))                          # [B, H, N, d]
    cu, lengths = s["cu"].long(), s["lengths"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(m, device=cu.device)
    row = (cu[:-1, None] + i).clamp(max=max(0, s["rows"] - 1))                        # [B, m]
    q = s["q"].float()[row].unflatten(2, (hkv, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)   # [B, H, m * G, d]
    z = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    last = lengths[:, None] - n[:, None] + i                                          # the last position that a query sees
    at = torch.arange(z.shape[-1], device=cu.device)
    seen = (at <= last[..., None]) & (at < lengths[:, None, None])
    if c["window"]:
        seen &= at > last[..., None] - c["window"]
    seen = seen[:, None].repeat_interleave(group, dim=2)
    z = z.masked_fill(~seen, -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    v = torch.where((at < lengths[:, None])[:, None, :, None], v, torch.zeros((), device=v.device))
    o = torch.matmul(p, v) / total.clamp(min=1e-30)
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(total, -math.inf))
    o = o.unflatten(2, (m, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)               # [B, m, Hq, d]
    lse = lse[..., 0].unflatten(2, (m, group)).permute(0, 2, 1, 3).flatten(2, 3)
    is_row = i < n[:, None]
    return o[is_row].to(s["q"].dtype), lse[is_row]


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "rope":
        c = state["case"]
        return _rotate(state["x"].float(), state, c["interleaved"], c["inverse"]).to(state["x"].dtype)
    return _plain_append(state) if op == "append" else _plain_attention(state)


# ------------------------------------------------------------------ the definition in 64 bits
def _e4m3_values():
    """The 127 finite values >= 0 of E4M3, from its bits."""
    return [(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127]


def _exact_rotation(x, s, interleaved, inverse):
    y = x.double().clone()
    table, pairs = s["table"].double(), s["table"].shape[1]
    for j in range(pairs):
        cs = table[s["positions"][s["pair_axis"][j]].long(), j]
        w = torch.complex(cs[:, 0], -cs[:, 1] if inverse else cs[:, 1])[:, None]
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + pairs)
        z = torch.complex(x[:, :, a].double(), x[:, :, b].double()) * w
        y[:, :, a], y[:, :, b] = z.real, z.imag
    return y


def _exact_stored(x, gain, values):
    """The values that a row's codes and scales stand for."""
    blocks = x.unflatten(-1, (-1, 16))
    want = (blocks.abs().amax(-1) / 7 / gain.double()[:, None]).clamp(max=448.0)
    hi = torch.searchsorted(values, want).clamp(max=len(values) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = values[hi] - want, want - values[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    step = (values[pick] * gain.double()[:, None])[..., None]
    return torch.where(step > 0, (blocks / step).round().clamp(-7, 7) * step, torch.zeros_like(blocks)).flatten(-2)


def _exact_rows(s, b, h, upto, values):
    """K and V of the first `upto` positions of sequence b, head h, in 64 bits."""
    c = s["case"]
    page, d = c["page"], c["head_dim"]
    got = s["pages"][s["page_table"][b, :-(-upto // page)].long(), h]
    if c["kv"] != "int4":
        return got[:, 0].double().flatten(0, 1)[:upto], got[:, 1].double().flatten(0, 1)[:upto]
    got = got.flatten(0, 1)                                                            # [groups, 18 d]
    out = []
    for first, gain, by_row in ((0, s["k_gain"][h], True), (9 * d, s["v_gain"][h], False)):
        byte = got[:, first:first + 8 * d].long()
        code = torch.empty(len(got), 16 * d, dtype=torch.float64, device=got.device)
        code[:, 0::2], code[:, 1::2] = (byte % 16 - 8).double(), (byte // 16 - 8).double()
        scale = values[got[:, first + 8 * d:first + 9 * d].long()]
        scale = scale.reshape(-1, 16, d // 16) if by_row else scale.reshape(-1, d // 16, 16).transpose(1, 2)
        x = code.reshape(-1, 16, d // 16, 16) * scale[..., None] * gain.double()
        out.append(x.reshape(-1, d)[:upto])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    device = s["table"].device if "table" in s else s["pages"].device
    if case["op"] == "rope":
        return _exact_rotation(s["x"], s, case["interleaved"], case["inverse"])
    values = torch.tensor(_e4m3_values() + [0.0], dtype=torch.float64, device=device)
    if case["op"] == "append":
        k, v = _exact_rotation(s["k"], s, False, False), s["v"].double()
        if case["kv"] == "int4":
            return _exact_stored(k, s["k_gain"], values[:127]), _exact_stored(v, s["v_gain"], values[:127])
        pages, page = s["pages"].double(), case["page"]
        lens, n = _counts(case)
        row = 0
        for b in range(case["batch"]):
            at = torch.arange(lens[b] - n[b], lens[b], device=device)
            pg = s["page_table"][b].long()[at // page]
            pages[pg, :, 0, at % page], pages[pg, :, 1, at % page] = k[row:row + n[b]], v[row:row + n[b]]
            row += n[b]
        return pages
    lens, n = _counts(case)
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    group = hq // hkv
    out = torch.zeros(sum(n), hq, d, dtype=torch.float64, device=device)
    lse = torch.full((sum(n), hq), -math.inf, dtype=torch.float64, device=device)
    row = 0
    for b in range(case["batch"]):
        for h in range(hkv if lens[b] and n[b] else 0):
            k, v = _exact_rows(s, b, h, lens[b], values)
            for i in range(n[b]):
                end = lens[b] - n[b] + i + 1
                begin = max(0, end - case["window"]) if case["window"] else 0
                if end <= begin:
                    continue
                q = s["q"][row + i, h * group:(h + 1) * group].double()
                z = (q @ k[begin:end].T) / math.sqrt(d)
                total = torch.logsumexp(z, dim=-1)
                out[row + i, h * group:(h + 1) * group] = torch.exp(z - total[:, None]) @ v[begin:end]
                lse[row + i, h * group:(h + 1) * group] = total
        row += n[b]
    return out, lse
