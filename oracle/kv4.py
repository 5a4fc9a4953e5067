"""The paged 4-bit cache in plain numpy and 64 bits: what page_plan, kv4_append, kv4_read and kv4_attn
compute, one request, row and token at a time.  Shares no code with the CUDA path."""
import numpy as np

DIM, GROUP = 512, 32
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E_MIN, E_MAX = -23, 13


def quantise(x):
    """x [n, DIM] (real) -> codes [n, DIM/2], scales [n, DIM/GROUP] uint8."""
    x = np.asarray(x, dtype=np.float64)
    n = x.shape[0]
    code = np.zeros((n, DIM), dtype=np.uint8)
    scale = np.zeros((n, DIM // GROUP), dtype=np.uint8)
    for g in range(DIM // GROUP):
        blk = x[:, g * GROUP:(g + 1) * GROUP]
        for r in range(n):
            v = blk[r]
            if np.isnan(v).any():
                scale[r, g] = 255
                continue                                       # its codes stand for nothing
            top = np.abs(v).max()
            e = E_MIN
            while e < E_MAX and top > 6.0 * 2.0 ** e:
                e += 1
            scale[r, g] = e + 127
            with np.errstate(invalid="ignore"):
                y = np.minimum(np.abs(v) * 2.0 ** -e, 6.0)
            dist = np.abs(y[:, None] - GRID[None, :])
            best = dist.min(axis=1, keepdims=True)
            tied = dist == best
            pick = tied.argmax(axis=1)                          # the lower of two tied codes
            upper = np.minimum(pick + 1, 7)
            two = tied.sum(axis=1) == 2
            pick = np.where(two & (pick % 2 == 1), upper, pick)  # ties go to the even code
            code[r, g * GROUP:(g + 1) * GROUP] = pick | (np.signbit(v).astype(np.uint8) << 3)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8), scale


def values(codes, scales):
    """codes [n, DIM/2], scales [n, DIM/GROUP] -> the float64 values they stand for."""
    codes = np.asarray(codes)
    nib = np.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=np.int64)
    nib[..., 0::2], nib[..., 1::2] = codes & 15, codes >> 4
    v = np.where(nib & 8, -1.0, 1.0) * GRID[nib & 7]
    s = np.where(np.asarray(scales) == 255, np.nan, 2.0 ** (np.asarray(scales, dtype=np.float64) - 127))
    return v * np.repeat(s, GROUP, axis=-1)


def page_plan(seen, n_new, rows, tables, free_pages, n_free, ratio, page_rows, T_cap, R_cap):
    """Returns (positions, req, slots, tables, seen_out, rows_out, n_free_out, totals)."""
    big = 2 ** 31 - 1
    B, max_pages = tables.shape
    tables = tables.copy()
    free = [int(x) for x in free_pages[:max(0, min(int(n_free), len(free_pages)))]]
    F = len(free)
    positions, req, slots, seen_out, rows_out = [], [], [], [], []
    tok = done_all = placed_all = 0
    for b in range(B):
        s = max(0, int(seen[b]))
        after = min(s + max(0, int(n_new[b])), big)
        take = min(after - s, max(0, T_cap - len(positions)))
        positions += range(s, s + take)
        req += [b] * take
        tok += after - s
        r = min(max(0, int(rows[b])), max_pages * page_rows)
        done = after // ratio - s // ratio
        done_all += done
        end = min(r + done, max_pages * page_rows)
        if r < s // ratio:                                           # it ran short earlier: row r is pooled row r
            end = r
        for pg in range(-(-r // page_rows), -(-end // page_rows)):   # new pages
            if not free:
                end = min(end, pg * page_rows)
                break
            tables[b, pg] = free.pop()
        for i in range(min(done, max(0, R_cap - len(slots)))):
            slot = -1
            if r + i < end:
                page = int(tables[b, (r + i) // page_rows])
                if page >= 0 and page * page_rows + (r + i) % page_rows <= big:
                    slot = page * page_rows + (r + i) % page_rows
            slots.append(slot)
        placed_all += end - r
        seen_out.append(after)
        rows_out.append(end)
    pad = lambda v, n: np.array(v + [-1] * (n - len(v)), dtype=np.int32)  # noqa: E731
    totals = np.array([min(tok, big), min(done_all, big), min(placed_all, big), F - len(free)], dtype=np.int32)
    return (pad(positions, T_cap), pad(req, T_cap), pad(slots, R_cap), tables, np.array(seen_out, dtype=np.int32),
            np.array(rows_out, dtype=np.int32), np.int32(len(free)), totals)


def attended_slots(t, tables, rows, page_rows, n_slots, req=None, positions=None, ratio=1, indices=None, counts=None):
    """Slots of the rows token t attends to, in list order."""
    b = t if req is None else int(req[t])
    if not 0 <= b < len(rows):
        return []
    held = min(max(0, int(rows[b])), tables.shape[1] * page_rows)
    if indices is not None:
        n = indices.shape[1] if counts is None else min(max(0, int(counts[t])), indices.shape[1])
        want = [int(r) for r in indices[t, :n] if 0 <= r < held]
    else:
        n = held if positions is None else min(held, (int(positions[t]) + 1) // ratio if positions[t] >= 0 else 0)
        want = range(n)
    out = []
    for r in want:
        page = int(tables[b, r // page_rows])
        slot = page * page_rows + r % page_rows
        if page >= 0 and slot < n_slots:
            out.append(slot)
    return out


def attn(q, pool, scale, **lists):
    """q [T, H, DIM] real, pool [n_slots, DIM] real values.  Returns out [T, H, DIM], lse [T, H] (float64)."""
    T, H, D = q.shape
    out = np.zeros((T, H, D))
    lse = np.full((T, H), -np.inf)
    for t in range(T):
        at = attended_slots(t, n_slots=pool.shape[0], **lists)
        if not at:
            continue
        kv = pool[at]
        x = (np.asarray(q[t], dtype=np.float64) @ kv.T) * scale
        m = x.max(axis=1, keepdims=True)
        p = np.exp(x - m)
        l = p.sum(axis=1, keepdims=True)
        out[t] = p @ kv / l
        lse[t] = (m + np.log(l))[:, 0]
    return out, lse
