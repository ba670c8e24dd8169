"""Operators around a paged cache: rotation of positions, 4-bit records, ragged attention.  Test infrastructure.

Plain numpy from the definitions in include/tkv.h, shares no code with the CUDA path.  What floating point decides
(a code, a scale byte) is decided in fp32 with the same operations as on the GPU, one rounding each; everything
else is fp64.
"""

import numpy as np

from . import fp8

F32 = np.float32


def rotate(x, table, positions, pair_axis, interleaved=False, inverse=False):
    """x fp32 [rows, heads, d] -> fp32, each product and each sum rounded once."""
    x = np.asarray(x, F32)
    y = x.copy()
    for j in range(table.shape[1]):
        p = positions[pair_axis[j]]
        c, s = table[p, j, 0][:, None], table[p, j, 1][:, None]
        s = -s if inverse else s
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + table.shape[1])
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y


def quantise(x, gain):
    """One head's row, fp32 [d] -> (codes q [d] int, scale bytes [d/16])."""
    x, gain = np.asarray(x, F32), F32(gain)
    q, b = np.zeros(len(x), int), np.zeros(len(x) // 16, np.uint8)
    for i in range(len(b)):
        blk = x[16 * i:16 * i + 16]
        if not np.all(np.isfinite(blk)):
            b[i] = 0x7F
            continue
        with np.errstate(over="ignore"):
            want = np.max(np.abs(blk)) / F32(F32(7) * gain)
        b[i] = fp8.encode(np.minimum(want, F32(448)))
        step = F32(fp8.DECODE_TABLE[b[i]]) * gain
        if step > 0:
            with np.errstate(over="ignore"):
                q[16 * i:16 * i + 16] = np.clip(np.rint(blk / step), -7, 7).astype(int)
    return q, b


def record_offsets(d):
    return 0, 8 * d, 9 * d, 17 * d


def put(record, r, which, q, b, d):
    """Writes position r of a record (uint8 [18 d]); which: 0 = K, 1 = V."""
    kc, ks, vc, vs = record_offsets(d)
    c = (np.asarray(q) + 8).astype(np.uint8)
    at = (vc if which else kc) + r * (d // 2)
    record[at:at + d // 2] = c[0::2] | (c[1::2] << 4)
    for i in range(d // 16):
        record[vs + 16 * i + r if which else ks + r * (d // 16) + i] = b[i]


def get(record, r, which, d, gain):
    """fp64 values of position r of a record."""
    kc, ks, vc, vs = record_offsets(d)
    at = (vc if which else kc) + r * (d // 2)
    c = record[at:at + d // 2].astype(int)
    q = np.stack([c & 15, c >> 4], axis=1).reshape(-1) - 8
    b = np.array([record[vs + 16 * i + r if which else ks + r * (d // 16) + i] for i in range(d // 16)])
    return q * np.repeat(fp8.DECODE_TABLE[b], 16) * np.float64(F32(gain))


def row_place(cu, lengths, page_table, page_size, num_pages, row):
    """(sequence, position, page, offset) of a step's row; page None: it has no place; None: behind the last."""
    b = int(np.searchsorted(cu, row, side="right")) - 1
    if b >= len(lengths):
        return None
    pos = int(lengths[b]) - (int(cu[b + 1]) - row)
    if pos < 0 or pos // page_size >= page_table.shape[1]:
        return b, pos, None, None
    page = int(page_table[b, pos // page_size])
    return b, pos, page if 0 <= page < num_pages else None, pos % page_size


def read(pages, page, off, h, d, k_gain=None, v_gain=None):
    """(K, V) fp64 [d] of one place of a pool: 4-bit records (uint8) or 16-bit rows given as floats."""
    if pages.dtype == np.uint8:
        rec = pages[page, h, off // 16]
        return tuple(get(rec, off % 16, i, d, 1.0 if g is None else g[h]) for i, g in ((0, k_gain), (1, v_gain)))
    return pages[page, h, 0, off].astype(np.float64), pages[page, h, 1, off].astype(np.float64)


def attend(q, pages, page_table, lengths, cu, page_size, hkv, window=0, scale=None, k_gain=None, v_gain=None):
    """fp64 (out [rows, Hq, d], lse [rows, Hq], A, S, F): A = sum of alpha |v|, S = the largest sum over channels of
    |q k| of a row and F = the positions it sees times their largest |v|, which the error bounds of the 16-bit products
    go by.  Rows behind the last: NaN."""
    rows, hq, d = q.shape
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    out, lse = np.full((rows, hq, d), np.nan), np.full((rows, hq), np.nan)
    absv, big, far = np.zeros((rows, hq, d)), np.zeros((rows, hq)), np.zeros((rows, hq))
    G = hq // hkv
    for b in range(len(lengths)):
        n, ln = int(cu[b + 1] - cu[b]), int(lengths[b])
        if n == 0:
            continue
        cap = min(ln, page_table.shape[1] * page_size)
        places = [(p, int(page_table[b, p // page_size])) for p in range(cap)]
        places = [(p, pg) for p, pg in places if 0 <= pg < pages.shape[0]]
        at = np.array([p for p, _ in places], int)
        for h in range(hkv):
            kv = [read(pages, pg, p % page_size, h, d, k_gain, v_gain) for p, pg in places]
            K = np.array([x[0] for x in kv]).reshape(-1, d)
            V = np.array([x[1] for x in kv]).reshape(-1, d)
            for i in range(n):
                last = ln - n + i
                see = (at <= last) & ((at > last - window) if window else True)
                for g in range(h * G, (h + 1) * G):
                    row = int(cu[b]) + i
                    if not np.any(see):
                        out[row, g], lse[row, g] = 0.0, -np.inf
                        continue
                    z = scale * (K[see] @ q[row, g])
                    m = z.max()
                    p = np.exp(z - m)
                    lse[row, g] = m + np.log(p.sum())
                    out[row, g] = (p / p.sum()) @ V[see]
                    absv[row, g] = (p / p.sum()) @ np.abs(V[see])
                    far[row, g] = len(z) * np.abs(V[see]).max()
                    big[row, g] = abs(scale) * (np.abs(K[see]) @ np.abs(q[row, g])).max()
    return out, lse, absv, big, far
