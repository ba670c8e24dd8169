"""Operators around a paged KV cache held in 8 bits, and beam search over paged caches: what is measured of them, and their plain forms.

  append     rows of k and v into 8-bit pages, k rotated on the way, a scale a block of 16 positions and head; read back by `gather`
  attention  the queries of a step over a paged cache held in 8 bits
  select     the best continuations of every sequence's beams, over beams and vocabulary
  reorder    the paged caches of all layers follow the beams that were chosen

The plain forms are elementary torch operations in 32 bits, in 64 where scores of candidates are compared.  An 8-bit page holds,
per KV head, records of 16 positions: K codes [d/64][16][64] | V codes [2][d/8][4][8][2] (half of the positions, channels / 8, pair of
positions, channel, position of the pair) | the exponents of K and of V, int32 | 8 bytes of zeros.  A value is E4M3(code) * 2^exponent.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
WIDTH = {"bf16": 2.0, "fp16": 2.0, "fp32": 4.0, "e4m3": 1.0, "int4": 0.5625}
LOWEST, HIGHEST = -32, 31   # exponents of a block


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step: one token a sequence, into blocks that hold tokens already
        dict(name="append_decode", op="append", dtype="bf16", batch=8, kv_heads=8, head_dim=128, page=64, prior=4099, new=1, axes=1),
        # prompts of several lengths enter the cache together
        dict(name="append_prompts", op="append", dtype="bf16", batch=8, kv_heads=8, head_dim=128, page=64, prior=301, new=4096, axes=1),
        # drafted tokens of many short sequences, small heads, an odd number of them, three axes
        dict(name="append_drafts_d64", op="append", dtype="fp16", batch=67, kv_heads=5, head_dim=64, page=16, prior=1531, new=6, axes=3),
        # batch 1, one reasoning chain of 2,512 positions, 28/4 heads
        dict(name="attend_one_chain", op="attention", dtype="bf16", batch=1, q_heads=28, kv_heads=4, head_dim=128, page=16, length=2512,
             ragged=False, new=1, window=0),
        # batch 8, 64/8 heads, 16,384 positions a sequence
        dict(name="attend_batch", op="attention", dtype="bf16", batch=8, q_heads=64, kv_heads=8, head_dim=128, page=64, length=16384,
             ragged=False, new=1, window=0),
        # the largest: a serving batch of mixed lengths up to 65,536, empty and idle sequences among them
        dict(name="attend_serving", op="attention", dtype="bf16", batch=32, q_heads=64, kv_heads=8, head_dim=128, page=64, length=65536,
             ragged=True, new=1, window=0),
        # several drafted tokens a sequence, small heads, an odd group, a window
        dict(name="attend_drafts_d64", op="attention", dtype="fp16", batch=19, q_heads=24, kv_heads=8, head_dim=64, page=32, length=6007,
             ragged=True, new=5, window=1000),
        # one sequence of four beams: what a launch costs
        dict(name="select_one", op="select", dtype="bf16", batch=1, beams=4, vocab=32000, count=8, finished=False),
        # an odd vocabulary in 32 bits, five beams, some of them finished
        dict(name="select_finished_fp32", op="select", dtype="fp32", batch=16, beams=5, vocab=100003, count=5, finished=True),
        # a large batch: 64 sequences of eight beams
        dict(name="select_batch", op="select", dtype="bf16", batch=64, beams=8, vocab=131072, count=16, finished=False),
        # 28 layers of 16-bit pages follow four beams
        dict(name="reorder_one", op="reorder", kv="bf16", layers=28, batch=1, beams=4, kv_heads=4, head_dim=128, page=16, length=2505),
        # 80 layers of 8-bit pages follow eight times eight beams
        dict(name="reorder_batch", op="reorder", kv="e4m3", layers=80, batch=8, beams=8, kv_heads=8, head_dim=128, page=64, length=1000),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "select", "reorder"])
    head_dim, page, kv_heads = rng.choice([64, 128]), rng.choice([16, 32, 64, 128]), rng.randint(1, 8)
    dtype = rng.choice(["bf16", "fp16"])
    if op == "append":
        batch = _log(rng, 1, 128)
        new = max(1, min(_log(rng, 1, 4096), 16384 // batch))
        return dict(op=op, dtype=dtype, batch=batch, kv_heads=kv_heads, head_dim=head_dim, page=page, prior=rng.randint(0, 4096),
                    new=new, axes=rng.randint(1, 3))
    if op == "attention":
        batch, group = _log(rng, 1, 128), rng.randint(1, 8)
        length = max(1, min(_log(rng, 1, 65536), int(1.4e9 / (batch * kv_heads * head_dim * 2))))
        new = min(length, rng.choice([1, 1, 1, rng.randint(2, 8)]))
        return dict(op=op, dtype=dtype, batch=batch, q_heads=group * kv_heads, kv_heads=kv_heads, head_dim=head_dim, page=page,
                    length=length, ragged=rng.random() < 0.7, new=new, window=rng.choice([0, 0, rng.randint(1, length)]))
    if op == "select":
        beams, batch = rng.randint(1, 16), _log(rng, 1, 64)
        vocab = max(16, min(_log(rng, 1000, 200000), (1 << 26) // (batch * beams)))
        return dict(op=op, dtype=rng.choice(["bf16", "fp16", "fp32"]), batch=batch, beams=beams, vocab=vocab,
                    count=rng.choice([beams, 2 * beams]), finished=rng.random() < 0.4)
    kv, beams = rng.choice(["e4m3", "e4m3", "int4", dtype]), rng.randint(2, 16)
    page_bytes = kv_heads * page * 2 * head_dim * WIDTH[kv]
    layers = max(1, min(_log(rng, 1, 80), int(6.5e8 / (beams * page_bytes))))
    batch = max(1, min(_log(rng, 1, 16), int(6.5e8 / (layers * beams * page_bytes))))
    return dict(op=op, kv=kv, layers=layers, batch=batch, beams=beams, kv_heads=kv_heads, head_dim=head_dim, page=page,
                length=_log(rng, 1, 2048))


def _counts(case):
    """(positions after the step, tokens of the step) of each sequence: a rule of the case alone."""
    b = case["batch"]
    if case["op"] == "append":   # the first sequence has `new` tokens, the others fewer
        n = [max(1, case["new"] * (b - i) // b) for i in range(b)]
        return [(case["prior"] * (i + 1)) // b + n[i] for i in range(b)], n
    new = case["new"]
    if not case["ragged"]:
        return [case["length"]] * b, [new] * b
    lens, n = [], []
    for i in range(b):           # the first is the longest; one in eleven is empty, one in seven idle
        f = 1.0 if i == 0 else (0.02 + 0.98 * ((i * 0.6180339887498949) % 1.0)) ** 2
        lens.append(0 if i % 11 == 7 else max(1, int(case["length"] * f)))
        n.append(0 if i % 7 == 5 else 1 + (new - 1 + 3 * i) % new)
    return lens, n


def _beam_lengths(case):
    """Positions of each sequence of beams: between three quarters of the longest and all."""
    return [max(1, case["length"] - (case["length"] // 4) * g // case["batch"]) for g in range(case["batch"])]


def _used(case, length):
    """Bytes of a position's K and V in the partly filled page that a reorder copies: what the format stores of it."""
    d, rest = case["head_dim"], length % case["page"]
    if case["kv"] == "e4m3":
        return -(-rest // 16) * (32 * d + 16)
    if case["kv"] == "int4":
        return -(-rest // 16) * 18 * d
    return rest * 2 * d * 2


def work(case):
    op = case["op"]
    if op == "select":
        n = case["batch"] * case["beams"]
        return {"bytes": n * (case["vocab"] * WIDTH[case["dtype"]] + 4) + case["batch"] * case["count"] * 12, "flops": 4 * n * case["vocab"]}
    if op == "reorder":
        w = case["beams"]
        moved = w * (1 - 1 / w)                               # beams that go on from another one, as expected of random parents
        read = w * (1 - (1 - 1 / w) ** w) * (1 - 1 / w)       # and the different ones that these go on from
        lens = _beam_lengths(case)
        rows = sum(_used(case, x) for x in lens) * case["kv_heads"] * case["layers"]
        columns = sum(x // case["page"] for x in lens)
        return {"bytes": (moved + read) * (rows + 4 * columns) + 4 * w * case["batch"], "flops": 0}
    lens, n = _counts(case)
    d, hkv = case["head_dim"], case["kv_heads"]
    if op == "append":
        t, back = sum(n), sum(m + (l - m) % 16 for l, m in zip(lens, n))
        return {"bytes": 2 * hkv * d * (t * (2 + 1) + back * (1 + 2)) + t * (d * 4 + 4 * case["axes"]), "flops": 3 * t * hkv * d}
    w0 = case["window"]
    seen = [0 if not m else l if not w0 else min(l, w0 + m - 1) for l, m in zip(lens, n)]
    pairs = sum(min(max(0, l - m + i + 1), w0 or l) for l, m in zip(lens, n) for i in range(m))
    return {"bytes": sum(seen) * hkv * (2 * d + 1) + sum(n) * case["q_heads"] * (d * 4 + 4), "flops": 4 * case["q_heads"] * d * pairs}


# ------------------------------------------------------------------ the 8-bit format
def _exponents(amax):
    """The least e with amax <= 448 * 2^e, within the format's range."""
    mantissa, e = torch.frexp(amax)
    e = e - 9 + (mantissa > 0.875).to(e.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, LOWEST)).clamp(LOWEST, HIGHEST)


def _power(e):
    """2^e in 32 bits, exactly: torch.ldexp and torch.pow round."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _amax(x):
    """The largest |x| of a block [..., 16, d] over what is finite."""
    return torch.where(torch.isfinite(x), x.abs(), torch.zeros((), device=x.device)).amax((-1, -2))


def _codes(x, e):
    """E4M3 bytes of x [..., 16, d] with the exponents e [...]; an infinity or a NaN is a NaN."""
    y = x * _power(-e)[..., None, None]
    q = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.where(torch.isfinite(x), q, torch.full_like(q, 0x7F))


def _values(codes, e):
    return codes.contiguous().view(torch.float8_e4m3fn).float() * _power(e)[..., None, None]


def _k_places(codes):
    """[..., 16, d] in the order of the record."""
    return codes.unflatten(-1, (-1, 64)).transpose(-3, -2).flatten(-3)


def _k_rows(rec, d):
    return rec.unflatten(-1, (d // 64, 16, 64)).transpose(-3, -2).flatten(-2)


def _v_places(codes):
    x = codes.unflatten(-1, (-1, 8)).unflatten(-3, (2, 4, 2))                            # half, pair, position, chunk, channel
    return x.movedim(-2, -4).movedim(-2, -1).flatten(-5)                               # half, chunk, pair, channel, position


def _v_rows(rec, d):
    x = rec.unflatten(-1, (2, d // 8, 4, 8, 2))
    return x.movedim(-1, -2).movedim(-4, -2).flatten(-5, -3).flatten(-2)


def _record(k_codes, v_codes, ke, ve):
    tail = torch.stack([ke, ve, torch.zeros_like(ke), torch.zeros_like(ke)], dim=-1).to(torch.int32).contiguous().view(torch.uint8)
    return torch.cat([_k_places(k_codes), _v_places(v_codes), tail], dim=-1)


def _tail(rec, d):
    """The exponents of records [..., 32 d + 16]."""
    e = rec[..., 32 * d:32 * d + 8].contiguous().view(torch.int32).clamp(LOWEST, HIGHEST)
    return e[..., 0], e[..., 1]


def _read(rec, d):
    """Records [..., 32 d + 16] -> K, V fp32 [..., 16, d]."""
    ke, ve = _tail(rec, d)
    return _values(_k_rows(rec[..., :16 * d], d), ke), _values(_v_rows(rec[..., 16 * d:32 * d], d), ve)


# ------------------------------------------------------------------ inputs
def _table(max_positions, pairs, device):
    freq = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device=device) / pairs)
    angle = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.stack([angle.cos(), angle.sin()], dim=-1).float().contiguous()


def _pool(g, lens, page, device, spare=2):
    """The pages of sequences of these lengths, in no order: the number of pages and the page table."""
    need = [max(1, -(-x // page)) for x in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=g, device=device).to(torch.int32)
    starts = [sum(need[:i]) for i in range(len(need))]
    cols = torch.arange(max(need), device=device)
    first, many = torch.tensor(starts, device=device)[:, None], torch.tensor(need, device=device)[:, None]
    return total, torch.where(cols < many, order[(first + cols).clamp(max=total - 1)], torch.zeros_like(order[:1])).contiguous()


def _fill(g, case, lens, device):
    """A cache whose rows are keys and values as a model makes them: normal, one position in a hundred a heavy hitter whose key lies
    along its head's direction u, one channel in 64 four times as large."""
    hkv, d, page = case["kv_heads"], case["head_dim"], case["page"]
    total, table = _pool(g, lens, page, device)
    u = torch.randn(hkv, d, generator=g, device=device)
    u = u / u.norm(dim=-1, keepdim=True)
    loud = torch.where(torch.rand(hkv, 1, d, generator=g, device=device) < 1 / 64, 4.0, 1.0)
    pages = torch.empty(total, hkv, page // 16, 32 * d + 16, dtype=torch.uint8, device=device)
    chunk = max(1, (1 << 26) // (hkv * page * d))
    for p in range(0, total, chunk):
        m = min(chunk, total - p)
        k = torch.randn(m, hkv, page, d, generator=g, device=device) * loud
        hot = torch.rand(m, 1, page, 1, generator=g, device=device) < 0.01
        k += torch.where(hot, 4.0, 0.0) * u[:, None]
        v = torch.randn(m, hkv, page, d, generator=g, device=device)
        k, v = (x.unflatten(2, (-1, 16)) for x in (k, v))
        ke, ve = _exponents(_amax(k)), _exponents(_amax(v))
        pages[p:p + m] = _record(_codes(k, ke), _codes(v, ve), ke, ve)
    return {"pages": pages, "page_table": table, "lengths": torch.tensor(lens, dtype=torch.int32, device=device), "u": u}


def _offsets(n, device):
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    return torch.tensor(cu, dtype=torch.int32, device=device)


def _prepare_select(case, g, device):
    b, w, v = case["batch"], case["beams"], case["vocab"]
    logits = torch.randn(b, w, v, generator=g, device=device) * 2.5          # many small ones, and in one beam of two a clear favourite
    best = torch.randint(0, v, (b, w, 1), generator=g, device=device)
    logits.scatter_add_(2, best, 14.0 * (torch.rand(b, w, 1, generator=g, device=device) < 0.5))
    s = {"logits": logits.to(DTYPES[case["dtype"]]),
         "scores": -(torch.rand(b, w, generator=g, device=device) * 10).sort(dim=-1)[0].contiguous(), "finished": None, "eos": None}
    if case["finished"]:
        s["finished"], s["eos"] = torch.rand(b, w, generator=g, device=device) < 0.2, 2
    return s


def _prepare_reorder(case, g, device):
    w, page, hkv, d = case["beams"], case["page"], case["kv_heads"], case["head_dim"]
    lens = _beam_lengths(case)
    columns = -(-(max(lens) + 1) // page)
    table, at = [], 0
    for x in lens:                      # four fifths of a sequence are its prompt, whose full pages its beams share
        prompt = min(x // page, 4 * x // 5 // page)
        for _ in range(w):
            private = range(at + prompt, at + prompt + columns - prompt)
            table.append(list(range(at, at + prompt)) + list(private))
            at += columns - prompt
        at += prompt
        for row in table[-w:]:
            row[:prompt] = range(at - prompt, at)
    order = torch.randperm(at, generator=g, device=device).to(torch.int32)
    s = {"page_table": order[torch.tensor(table, device=device)].contiguous(),
         "lengths": torch.tensor([x for x in lens for _ in range(w)], dtype=torch.int32, device=device),
         "parents": torch.randint(0, w, (case["batch"], w), generator=g, device=device, dtype=torch.int32)}
    if case["kv"] in ("e4m3", "int4"):
        shape = (case["layers"], at, hkv, page // 16, 32 * d + 16 if case["kv"] == "e4m3" else 18 * d)
        s["pages"] = torch.randint(0, 120, shape, generator=g, device=device, dtype=torch.uint8)
    else:
        s["pages"] = torch.randn(case["layers"], at, hkv, 2, page, d, generator=g, device=device, dtype=DTYPES[case["kv"]])
    return s


def prepare(case, seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] in ("select", "reorder"):
        s.update((_prepare_select if case["op"] == "select" else _prepare_reorder)(case, g, device))
        return s
    lens, n = _counts(case)
    hkv, d = case["kv_heads"], case["head_dim"]
    s.update(_fill(g, case, lens, device))
    s["cu"], s["rows"], s["max_new"], s["max_len"] = _offsets(n, device), sum(n), max(n), max(lens)
    dt = DTYPES[case["dtype"]]
    if case["op"] == "append":
        t = s["rows"]
        back = [m + (l - m) % 16 for l, m in zip(lens, n)]   # what is read back: the blocks that the step touches
        s["cu_back"], s["rows_back"] = _offsets(back, device), sum(back)
        loud = torch.exp2(torch.randint(-1, 3, (t, 1, 1), generator=g, device=device).float())
        s["k"], s["v"] = ((torch.randn(t, hkv, d, generator=g, device=device) * loud).to(dt) for _ in range(2))
        _, pos = _where(s["cu"], s["lengths"], t)
        more = [torch.randint(0, 512, pos.shape, generator=g, device=device, dtype=torch.int32) for _ in range(case["axes"] - 1)]
        s["positions"] = torch.stack([pos.to(torch.int32)] + more).contiguous()
        s["table"] = _table(16384, d // 2, device)
        s["pair_axis"] = [j * case["axes"] // (d // 2) for j in range(d // 2)]
        s["axis_of_pair"] = torch.tensor(s["pair_axis"], device=device)
        return s
    group = case["q_heads"] // hkv
    q = torch.randn(s["rows"], hkv, group, d, generator=g, device=device) + 0.5 * math.sqrt(d) * s["u"][:, None]
    s["q"] = q.reshape(s["rows"], case["q_heads"], d).to(dt)
    return s


# ------------------------------------------------------------------ the framework's operators
def _handles(s):
    """The caches and the rotation that a user's program builds once."""
    import tiered_kv_cache_gqa_gb300 as tkv
    if "rotary" not in s and "table" in s:
        s["rotary"] = tkv.Rotary(s["table"], pair_axis=s["pair_axis"])
    if "cache" not in s and "pages" in s:
        if s["case"]["op"] == "reorder":
            s["cache"] = tkv.PagedLayers([tkv.PagedCache(p, s["page_table"], s["lengths"]) for p in s["pages"]])
        else:
            s["cache"] = tkv.PagedCache(s["pages"], s["page_table"], s["lengths"])
    return tkv


def _run_own(s):
    tkv, c = _handles(s), s["case"]
    if c["op"] == "select":
        return tkv.beam_select(s["logits"], s["scores"], count=c["count"], finished=s["finished"], eos=s["eos"])
    if c["op"] == "reorder":
        s["cache"].reorder(s["parents"])
        return s["page_table"], s["pages"]
    if c["op"] == "append":
        s["cache"].append(s["k"], s["v"], s["cu"], rotary=s["rotary"], positions=s["positions"])
        return s["cache"].gather(s["cu_back"], s["rows_back"], dtype=s["k"].dtype)
    return s["cache"].attend(s["q"], s["cu"], max_new=s["max_new"], max_len=s["max_len"], window=c["window"], return_lse=True)


# ------------------------------------------------------------------ the plain forms
def _rotate(x, s):
    """x fp32 [T, H, d], turned by halves."""
    pairs = s["table"].shape[1]
    at = s["positions"].long()[s["axis_of_pair"]].T                                  # [T, pairs]
    cs = s["table"][at, torch.arange(pairs, device=x.device)]                        # [T, pairs, 2]
    c, sn = cs[:, None, :, 0], cs[:, None, :, 1]
    x0, x1 = x[..., :pairs], x[..., pairs:]
    return torch.cat([x0 * c - x1 * sn, x1 * c + x0 * sn], dim=-1)


def _where(cu, lengths, rows):
    """The sequence and the position of each row of a step."""
    cu, lengths = cu.long(), lengths.long()
    row = torch.arange(rows, device=cu.device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    return seq, lengths[seq] - (cu[seq + 1] - row)


def _plain_append(s):
    page, d = s["case"]["page"], s["case"]["head_dim"]
    seq, pos = _where(s["cu"], s["lengths"], s["rows"])
    pg, off = s["page_table"].long()[seq, pos // page], pos % page
    first = (pos % 16 == 0) | (torch.arange(s["rows"], device=pos.device) == s["cu"].long()[seq])   # row of its block
    block = first.cumsum(0) - 1
    lead = first.nonzero()[:, 0]
    at = (pg[lead], off[lead] // 16, pos[lead] % 16)                                    # page, record, rows that are kept
    recs = s["pages"][at[0], :, at[1]]                                                  # [blocks, H, bytes]
    r = torch.arange(16, device=pos.device)
    new = torch.zeros(len(lead), 16, dtype=torch.bool, device=pos.device)
    new[block, pos % 16] = True
    new = new[:, None, :, None]
    kept = (r < at[2][:, None])[:, None, :, None]
    parts = []
    for x, rows_of, places, lo, which in ((_rotate(s["k"].float(), s), _k_rows, _k_places, 0, 0), (s["v"].float(), _v_rows, _v_places, 16 * d, 1)):
        old_codes, old = rows_of(recs[..., lo:lo + 16 * d], d), _tail(recs, d)[which]
        rows = torch.zeros(len(lead), 16, x.shape[1], d, device=x.device)
        rows[block, pos % 16] = x
        rows = rows.transpose(1, 2)                                                     # [blocks, H, 16, d]
        e = _exponents(_amax(rows))
        e = torch.where((at[2] > 0)[:, None], torch.maximum(e, old), e)
        codes = torch.where(new, _codes(rows, e), torch.where(kept, _codes(_values(old_codes, old), e), old_codes))
        parts.append((places(codes), e))
    tail = torch.stack([parts[0][1], parts[1][1], torch.zeros_like(e), torch.zeros_like(e)], dim=-1).to(torch.int32).contiguous()
    s["pages"][at[0], :, at[1]] = torch.cat([parts[0][0], parts[1][0], tail.view(torch.uint8)], dim=-1)
    return _plain_gather(s)


def _plain_gather(s):
    page, d = s["case"]["page"], s["case"]["head_dim"]
    seq, pos = _where(s["cu_back"], s["lengths"], s["rows_back"])
    pg, rec, r = s["page_table"].long()[seq, pos // page], pos % page // 16, pos % 16
    ke, ve = _tail(s["pages"], d)
    k = s["pages"][..., :16 * d].unflatten(3, (d // 64, 16, 64))[pg, :, rec, :, r]         # [T, H, d / 64, 64]
    v = s["pages"][..., 16 * d:32 * d].unflatten(3, (2, d // 8, 4, 8, 2))[pg, :, rec, r // 8, :, r % 8 // 2, :, r % 2]
    k, v = (_values(x.flatten(2)[:, :, None], e[pg, :, rec])[:, :, 0] for x, e in ((k, ke), (v, ve)))
    return k.to(s["k"].dtype), v.to(s["k"].dtype)


def _plain_attention(s):
    c = s["case"]
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    group, m = hq // hkv, s["max_new"]
    k, v = _read(s["pages"][s["page_table"].long()], d)                                  # [B, P, H, records, 16, d]
    k, v = (x.transpose(1, 2).flatten(2, 4) for x in (k, v))                             # [B, H, N, d]
    cu, lengths = s["cu"].long(), s["lengths"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(m, device=cu.device)
    row = (cu[:-1, None] + i).clamp(max=max(0, s["rows"] - 1))                           # [B, m]
    q = s["q"].float()[row].unflatten(2, (hkv, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)   # [B, H, m * G, d]
    z = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    last = lengths[:, None] - n[:, None] + i                                             # the last position that a query sees
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
    o = o.unflatten(2, (m, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)                  # [B, m, Hq, d]
    lse = lse[..., 0].unflatten(2, (m, group)).permute(0, 2, 1, 3).flatten(2, 3)
    is_row = i < n[:, None]
    return o[is_row].to(s["q"].dtype), lse[is_row]


def _plain_select(s):
    """Totals in 64 bits: those of two beams may lie as near as their roundings."""
    x, scores, v = s["logits"].double(), s["scores"].double(), s["case"]["vocab"]
    top = x.amax(-1, keepdim=True)
    total = scores[..., None] + ((x - top) - torch.log(torch.exp(x - top).sum(-1, keepdim=True)))
    if s["finished"] is not None:
        eos = torch.arange(v, device=x.device) == s["eos"]
        total = torch.where(s["finished"][..., None], torch.where(eos, scores[..., None], -math.inf), total)
    total = total.masked_fill(total.isnan(), -math.inf).flatten(1)
    best, at = total.sort(dim=-1, descending=True, stable=True)                          # ties to the lowest place
    best, at = best[:, :s["case"]["count"]], at[:, :s["case"]["count"]]
    none = best == -math.inf
    return best.float(), (at // v).masked_fill(none, -1).to(torch.int32), (at % v).masked_fill(none, -1).to(torch.int32)


def _plain_reorder(s):
    c = s["case"]
    page, w = c["page"], c["beams"]
    table, lengths = s["page_table"].long(), s["lengths"].long()
    seq = torch.arange(len(lengths), device=table.device)
    parent = seq // w * w + s["parents"].flatten().long()
    current, rest = lengths // page, lengths % page
    own_page = table.gather(1, current[:, None])[:, 0]
    position = torch.arange(page, device=table.device)
    if c["kv"] in ("e4m3", "int4"):                                                       # whole records that hold a position
        held = (position[:page // 16] * 16 < rest[:, None])[None, :, None, :, None]
    else:
        held = (position < rest[:, None])[None, :, None, None, :, None]
    s["pages"][:, own_page] = torch.where(held, s["pages"][:, own_page[parent]], s["pages"][:, own_page])
    before = torch.arange(table.shape[1], device=table.device) < current[:, None]
    s["page_table"].copy_(torch.where(before, s["page_table"][parent], s["page_table"]))
    return s["page_table"], s["pages"]


def run(state):
    if own:
        return _run_own(state)
    plain = {"append": _plain_append, "attention": _plain_attention, "select": _plain_select, "reorder": _plain_reorder}
    return plain[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits
def _e4m3_values(device):
    """The 256 values of E4M3, from its bits."""
    low = [(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)]
    low[127] = math.nan
    return torch.tensor(low + [-x for x in low], dtype=torch.float64, device=device)


def _two_to(e):
    """2^e in 64 bits, exactly."""
    return torch.tensor([2.0 ** k for k in range(LOWEST, HIGHEST + 1)], dtype=torch.float64, device=e.device)[e.long() - LOWEST]


def _exact_stored(x, e, values):
    """The nearest value of the format (ties to the even code) of x, in 64 bits, with exponents e."""
    y = (x.abs() / _two_to(e)).clamp(max=448.0)
    grid = values[:127]
    hi = torch.searchsorted(grid, y).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - y, y - grid[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.where(x < 0, -1.0, 1.0) * grid[pick] * _two_to(e)


def _exact_scale(amax):
    scale = torch.full_like(amax, LOWEST)
    for e in range(LOWEST, HIGHEST):
        scale += amax > 448.0 * 2.0 ** e      # the least exponent that is large enough: one more for each that is not
    return scale


def _exact_read(rec, d, values):
    """Records [N, 32 d + 16] -> K, V [N, 16, d] and exponents, in 64 bits, place by place."""
    p, c = torch.arange(16, device=rec.device)[:, None], torch.arange(d, device=rec.device)
    k_at = (c // 64) * 1024 + p * 64 + c % 64
    v_at = 16 * d + (p // 8) * 8 * d + (c // 8) * 64 + (p % 8 // 2) * 16 + (c % 8) * 2 + p % 2
    e = rec[:, 32 * d:32 * d + 8].contiguous().view(torch.int32)
    return [values[rec[:, at.flatten()].long()].unflatten(1, (16, d)) * _two_to(e[:, i, None, None]) for i, at in ((0, k_at), (1, v_at))], e


def _exact_append(s, case, values):
    lens, n = _counts(case)
    page, d, hkv = case["page"], case["head_dim"], case["kv_heads"]
    k = torch.empty(s["rows"], hkv, d, dtype=torch.float64, device=values.device)
    x, table, half = s["k"].double(), s["table"].double(), d // 2
    for j in range(half):
        cs = table[s["positions"][s["pair_axis"][j]].long(), j]
        z = torch.complex(x[:, :, j], x[:, :, j + half]) * torch.complex(cs[:, 0], cs[:, 1])[:, None]
        k[:, :, j], k[:, :, j + half] = z.real, z.imag
    new = (k, s["v"].double())
    out, row = [], 0
    for b in range(case["batch"]):
        start = lens[b] - n[b]
        kept = start % 16
        at = torch.arange(start - kept, lens[b], device=values.device)
        padded = -(-(kept + n[b]) // 16) * 16
        pg = int(s["page_table"][b, start // page])
        old, e = _exact_read(s["pages"][pg, :, start % page // 16], d, values)
        both = []
        for i in range(2):
            y = torch.zeros(padded, hkv, d, dtype=torch.float64, device=values.device)
            y[kept:kept + n[b]] = new[i][row:row + n[b]]
            blocks = y.unflatten(0, (-1, 16))
            scale = _exact_scale(blocks.abs().amax((1, 3)))                                # [blocks, H]
            if kept:
                scale[0] = torch.maximum(scale[0], e[:, i])
                blocks[0, :kept] = old[i].transpose(0, 1)[:kept]
            both.append(_exact_stored(blocks, scale[:, None, :, None], values).flatten(0, 1)[:len(at)])
        out.append(both)
        row += n[b]
    return torch.cat([x[0] for x in out]), torch.cat([x[1] for x in out])


def _exact_attention(s, case, values):
    lens, n = _counts(case)
    hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    group = hq // hkv
    out = torch.zeros(sum(n), hq, d, dtype=torch.float64, device=values.device)
    lse = torch.full((sum(n), hq), -math.inf, dtype=torch.float64, device=values.device)
    row = 0
    for b in range(case["batch"]):
        for h in range(hkv if lens[b] and n[b] else 0):
            recs = s["pages"][s["page_table"][b, :-(-lens[b] // page)].long(), h].flatten(0, 1)
            k, v = (x.flatten(0, 1)[:lens[b]] for x in _exact_read(recs, d, values)[0])
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


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "select":
        best = []
        for b in range(case["batch"]):
            total = torch.log_softmax(s["logits"][b].double(), dim=-1) + s["scores"][b].double()[:, None]
            if s["finished"] is not None:
                total[s["finished"][b]] = -math.inf
                total[s["finished"][b], s["eos"]] = s["scores"][b][s["finished"][b]].double()
            best.append(total.flatten().topk(case["count"])[0])
        return torch.stack(best), None, None
    if case["op"] == "reorder":
        if case["kv"] in ("e4m3", "int4"):
            return None
        pages, lens, w = s["pages"].double(), _beam_lengths(case), case["beams"]
        before = pages.clone()
        for g in range(case["batch"]):
            column, rest = lens[g] // case["page"], lens[g] % case["page"]
            for i in range(w if rest else 0):
                to, p = int(s["page_table"][g * w + i, column]), int(s["parents"][g, i])
                pages[:, to, :, :, :rest] = before[:, int(s["page_table"][g * w + p, column]), :, :, :rest]
        return None, pages
    values = _e4m3_values(s["pages"].device)
    return _exact_append(s, case, values) if case["op"] == "append" else _exact_attention(s, case, values)
