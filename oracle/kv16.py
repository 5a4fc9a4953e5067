"""The paged 16-bit cache in plain numpy and 64 bits: what rotate, kv16_append and kv16_attn compute, one row and
token at a time.  Shares no code with the CUDA path."""
import numpy as np


def rotate(x, positions, inv_freq, inverse=False):
    """x [T, ..., D] real -> float64, the last 2 len(inv_freq) elements of each row turned by its token's position."""
    y = np.array(x, dtype=np.float64)
    f = np.asarray(inv_freq, dtype=np.float64)
    start = y.shape[-1] - 2 * len(f)
    for t in range(y.shape[0]):
        a = int(positions[t]) * f
        if inverse:
            a = -a
        for i in range(len(f)):
            k = start + 2 * i
            x0, x1 = y[t, ..., k].copy(), y[t, ..., k + 1].copy()
            y[t, ..., k] = x0 * np.cos(a[i]) - x1 * np.sin(a[i])
            y[t, ..., k + 1] = x1 * np.cos(a[i]) + x0 * np.sin(a[i])
    return y


def seen_rows(t, tables, rows, page_rows, n_slots, req=None, positions=None, ratio=1, window=0, first=None, prefix=None):
    """(e, row numbers, slots) of the rows that token t sees."""
    b = t if req is None else int(req[t])
    if not 0 <= b < len(rows):
        return 0, [], []
    held = min(max(0, int(rows[b])), tables.shape[1] * page_rows)
    e = held
    if positions is not None:
        if positions[t] < 0:
            return 0, [], []
        e = (int(positions[t]) + 1) // ratio
    see, at = [], []
    for r in range(held):
        if not (r < e or (prefix is not None and r < int(prefix[b]))):
            continue
        if (window and r < e - window) or (first is not None and r < int(first[t])):
            continue
        page = int(tables[b, r // page_rows])
        slot = page * page_rows + r % page_rows
        if page >= 0 and slot < n_slots:
            see.append(r)
            at.append(slot)
    return e, see, at


def logits(q, kv, see, e, scale, cap=0.0, slopes=None):
    """q [H, D], kv [n, D] -> [H, n]."""
    x = np.asarray(q, dtype=np.float64) @ kv.T * scale
    if cap:
        x = cap * np.tanh(x / cap)
    if slopes is not None:
        x = x - np.asarray(slopes, dtype=np.float64)[:, None] * np.abs(e - 1 - np.asarray(see, dtype=np.int64))[None, :]
    return x


def attn(q, pool, scale, cap=0.0, slopes=None, sinks=None, other=None, **lists):
    """q [T, H, D] real, pool [n_slots, D] real.  Returns out [T, H, D], lse [T, H] (float64)."""
    T, H, D = q.shape
    out = np.zeros((T, H, D))
    lse = np.full((T, H), -np.inf)
    for t in range(T):
        e, see, at = seen_rows(t, n_slots=pool.shape[0], **lists)
        terms = [np.zeros((H, 0)), ]
        if see:
            terms = [logits(q[t], pool[at], see, e, scale, cap, slopes)]
        if sinks is not None:
            terms.append(np.asarray(sinks, dtype=np.float64)[:, None])
        if other is not None:
            terms.append(np.asarray(other[1][t], dtype=np.float64)[:, None])
        x = np.concatenate(terms, axis=1)
        if x.shape[1] == 0:
            continue
        for h in range(H):
            m = x[h].max()
            if m == -np.inf:
                continue
            w = np.exp(x[h] - m)
            lse[t, h] = m + np.log(w.sum())
            p = w / w.sum()
            if see:
                out[t, h] = p[:len(see)] @ pool[at]
            if other is not None and p[-1] != 0:
                out[t, h] += p[-1] * np.asarray(other[0][t, h], dtype=np.float64)
    return out, lse
