"""Beam search over paged caches: the choice of continuations, and caches that follow it.  Test infrastructure.

Plain numpy in fp64 from the definitions in include/tkv.h, shares no code with the CUDA path.
"""

import numpy as np


def totals(logits, scores, finished=None, eos=None):
    """fp64 [batch, beams, vocab]: each candidate's total, -infinity where there is none."""
    x = np.asarray(logits, np.float64)
    out = np.full(x.shape, -np.inf)
    for b in range(x.shape[0]):
        for w in range(x.shape[1]):
            s = float(scores[b, w])
            if not np.isfinite(s):
                continue
            if finished is not None and finished[b, w]:
                out[b, w, eos] = s
                continue
            row = x[b, w]
            if np.isnan(row).any() or (row == np.inf).any() or not (row > -np.inf).any():
                continue
            top = row.max()
            out[b, w] = s + ((row - top) - np.log(np.exp(row - top).sum()))
    return out


def select(logits, scores, count, finished=None, eos=None):
    """(scores fp64, beams, tokens), each [batch, count]."""
    t = totals(logits, scores, finished, eos)
    batch, _, vocab = t.shape
    best, beams, tokens = np.full((batch, count), -np.inf), np.full((batch, count), -1), np.full((batch, count), -1)
    for b in range(batch):
        flat = t[b].reshape(-1)
        order = np.lexsort((np.arange(flat.size), -flat))[:count]   # descending; ties by place
        order = order[flat[order] > -np.inf]
        best[b, :len(order)], beams[b, :len(order)], tokens[b, :len(order)] = flat[order], order // vocab, order % vocab
    return best, beams, tokens


def reorder(tables, lengths, parents, page_size, caches):
    """The page table after a reordering and each cache's pages: caches are (pages, units of 16 positions or of 1), their pages
    [num_pages, Hkv, page_size / 16, bytes] (records) or [num_pages, Hkv, 2, page_size, d]."""
    groups, beams = parents.shape
    table, after = tables.copy(), [c.copy() for c in caches]
    for g in range(groups):
        seqs = [g * beams + w for w in range(beams)]
        n = int(lengths[seqs[0]])
        column, rest = n // page_size, n % page_size
        if any(int(lengths[s]) != n for s in seqs) or n < 0 or column + (rest > 0) > tables.shape[1]:
            continue
        for w, p in enumerate(parents[g]):
            if not 0 <= p < beams or p == w:
                continue
            child, parent = seqs[w], seqs[p]
            table[child, :column] = tables[parent, :column]
            if not rest:
                continue
            to, frm = int(tables[child, column]), int(tables[parent, column])
            for before, now in zip(caches, after):
                if not (0 <= to < len(before) and 0 <= frm < len(before)):
                    continue
                if before.ndim == 4:
                    now[to, :, :-(-rest // 16)] = before[frm, :, :-(-rest // 16)]
                else:
                    now[to, :, :, :rest] = before[frm, :, :, :rest]
    return table, after
