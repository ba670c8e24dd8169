"""8-bit pages of a paged cache: E4M3 records with one exponent for a block of 16 positions.  Test infrastructure.

Plain numpy from the definitions in include/tkv.h, shares no code with the CUDA path.  What floating point decides (a code, an
exponent) is decided in fp32 with one rounding; everything else is fp64.
"""

import numpy as np

from . import fp8

F32 = np.float32
LOWEST, HIGHEST = -32, 31


def record_bytes(d):
    return 32 * d + 16


def k_place(p, c, d):
    """The byte of K's channel c at position p of a record."""
    return (c // 64) * 1024 + p * 64 + c % 64


def v_place(p, c, d):
    return 16 * d + (p // 8) * 8 * d + (c // 8) * 64 + (p % 8 // 2) * 16 + (c % 8) * 2 + p % 2


def exponent(amax):
    """The least e with amax <= 448 * 2^e, within the format's range."""
    for e in range(LOWEST, HIGHEST):
        if float(amax) <= 448.0 * 2.0 ** e:
            return e
    return HIGHEST


def encode(x, e):
    """Codes of fp32 values with a block's exponent; what is not finite is NaN."""
    x = np.asarray(x, F32)
    fine = np.isfinite(x)
    y = np.where(fine, x, F32(0)).astype(np.float64) * 2.0 ** -e
    y = np.clip(y, -448.0, 448.0).astype(F32)   # exact: a power of two, and 448
    return np.where(fine, fp8.encode(y), 0x7F).astype(np.uint8)


def exponents(rec, d):
    """(e_k, e_v) of a record (uint8 [32 d + 16])."""
    e = rec[32 * d:32 * d + 8].copy().view(np.int32)
    return tuple(int(np.clip(x, LOWEST, HIGHEST)) for x in e)


def rows(rec, d):
    """(K, V) fp64 [16, d] of a record."""
    p, c = np.arange(16)[:, None], np.arange(d)
    ke, ve = exponents(rec, d)
    return fp8.DECODE_TABLE[rec[k_place(p, c, d)]] * 2.0 ** ke, fp8.DECODE_TABLE[rec[v_place(p, c, d)]] * 2.0 ** ve


def append_block(rec, first, k, v):
    """Rows k, v (fp32 [n, d]) into a record from offset `first` on; the rows before it are kept."""
    d = k.shape[1]
    old, c = rows(rec, d), np.arange(d)
    for which, (x, place) in enumerate(((k, k_place), (v, v_place))):
        a = np.abs(np.where(np.isfinite(x), x, F32(0))).max()
        e_new, e_old = exponent(a), exponents(rec, d)[which]
        e = e_new if first == 0 else max(e_new, e_old)
        if first and e > e_old:
            p = np.arange(first)[:, None]
            rec[place(p, c, d)] = encode(old[which][:first].astype(F32), e)
        p = np.arange(first, first + len(x))[:, None]
        rec[place(p, c, d)] = encode(x, e)
        if not first or e > e_old:
            rec[32 * d + 4 * which:32 * d + 4 * which + 4] = np.array([e], np.int32).view(np.uint8)


def append(pages, page_table, lengths, cu, page_size, k, v):
    """A step's rows (fp32 [rows, Hkv, d], k already rotated) into pages [num_pages, Hkv, page_size / 16, 32 d + 16]."""
    for b in range(len(lengths)):
        n, pos, row = int(cu[b + 1] - cu[b]), int(lengths[b] - (cu[b + 1] - cu[b])), int(cu[b])
        while n > 0:
            take = min(n, 16 - pos % 16)
            page = int(page_table[b, pos // page_size]) if 0 <= pos < page_table.shape[1] * page_size else -1
            if 0 <= page < pages.shape[0]:
                for h in range(pages.shape[1]):
                    append_block(pages[page, h, pos % page_size // 16], pos % 16, k[row:row + take, h], v[row:row + take, h])
            n, pos, row = n - take, pos + take, row + take


def sequence(pages, page_table, b, length, page_size, h):
    """(positions that exist, K, V fp64, the V exponents) of a sequence's head."""
    d = (pages.shape[3] - 16) // 32
    at, K, V, E = [], [], [], []
    for p0 in range(0, min(length, page_table.shape[1] * page_size), 16):
        page = int(page_table[b, p0 // page_size])
        if not 0 <= page < pages.shape[0]:
            continue
        rec = pages[page, h, p0 % page_size // 16]
        kr, vr = rows(rec, d)
        n = min(16, length - p0)
        at += range(p0, p0 + n)
        K.append(kr[:n])
        V.append(vr[:n])
        E += [exponents(rec, d)[1]] * n
    return np.array(at, int), np.concatenate(K or [np.zeros((0, d))]), np.concatenate(V or [np.zeros((0, d))]), np.array(E, int)


def attend(q, pages, page_table, lengths, cu, page_size, window=0, scale=None):
    """fp64 (out, lse, A, S, F) as paged.attend gives them; F: the positions a row sees times the largest number that a block it
    looks into can hold, 448 * 2^e_v."""
    nrows, hq, d = q.shape
    hkv = pages.shape[1]
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    out, lse = np.full((nrows, hq, d), np.nan), np.full((nrows, hq), np.nan)
    absv, big, far = np.zeros((nrows, hq, d)), np.zeros((nrows, hq)), np.zeros((nrows, hq))
    G = hq // hkv
    for b in range(len(lengths)):
        n, ln = int(cu[b + 1] - cu[b]), int(lengths[b])
        for h in range(hkv if n else 0):
            at, K, V, E = sequence(pages, page_table, b, ln, page_size, h)
            for i in range(n):
                row, last = int(cu[b]) + i, ln - n + i
                see = (at <= last) & ((at > last - window) if window else True)
                for g in range(h * G, (h + 1) * G):
                    if not np.any(see):
                        out[row, g], lse[row, g] = 0.0, -np.inf
                        continue
                    z = scale * (K[see] @ q[row, g])
                    m = z.max()
                    p = np.exp(z - m)
                    lse[row, g] = m + np.log(p.sum())
                    out[row, g] = (p / p.sum()) @ V[see]
                    absv[row, g] = (p / p.sum()) @ np.abs(V[see])
                    far[row, g] = len(z) * 448.0 * 2.0 ** E[see].max()
                    big[row, g] = abs(scale) * (np.abs(K[see]) @ np.abs(q[row, g])).max()
    return out, lse, absv, big, far
