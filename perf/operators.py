"""Cases and plain forms of the 4-bit paged cache operators.

  plan    page_plan: positions, request ids, block tables and slots of one step, from request lengths
  append  kv4_append, read back with kv4_read: pooled rows quantised into the paged cache
  read    kv4_read: rows of the cache as 16-bit values
  attn    kv4_attn: 64-head multi-query attention over selected or all visible rows of the cache

The cache holds a row as 4-bit e2m1 codes (element 2i in the low nibble of byte i) with one power-of-two
scale a group of 32, stored as the byte e + 127: value = code * 2^e.  e is the least exponent with
max|x| <= 6 * 2^e, kept in [-23, 13], where every value is exact in fp16 and in bf16.
"""
import math

import numpy as np
import torch

own = False

D, HQ, GROUP = 512, 64, 32
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
E_MIN, E_MAX = -23, 13
INT_MAX = 2**31 - 1


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of 64 running requests, one position each: latency
        dict(name="plan_decode_64", kind="plan", n_req=64, new_lo=1, new_hi=1, seen_hi=65536, ratio=4, page_rows=64),
        # a mixed step of a large server: 1500 requests, most with a prefill chunk, pages running short
        dict(name="plan_mixed_1500", kind="plan", n_req=1500, new_lo=0, new_hi=128, seen_hi=30000, ratio=4,
             page_rows=32),
        # the pooled rows one decode step of a batch completes
        dict(name="append_decode_16", kind="append", n=16, page_rows=64, dtype="bf16"),
        # the pooled rows of a long prefill batch (64k positions a request, ratio 4, several requests)
        dict(name="append_prefill_50001", kind="append", n=50001, page_rows=64, dtype="f16"),
        # the 512 selected rows of one token, and the rows of a request handed to a 16-bit path
        dict(name="read_512", kind="read", n=512, page_rows=64, dtype="bf16"),
        dict(name="read_65536", kind="read", n=65536, page_rows=16, dtype="f16"),
        # one decode token over its 512 selected rows of a 1M-token context
        dict(name="attn_decode_1", kind="attn", n_req=1, per_req=1, rows_lo=262144, rows_hi=262144, page_rows=64,
             k_top=512, ratio=4, dtype="bf16"),
        # a decode batch: contexts from a few rows (fewer than 512: shorter lists) to 64k rows
        dict(name="attn_decode_67", kind="attn", n_req=67, per_req=1, rows_lo=3, rows_hi=65536, page_rows=64,
             k_top=512, ratio=4, dtype="f16"),
        # a 2048-token prefill chunk at 8k, ratio 4: 512 selected of at most 2048 rows a token
        dict(name="attn_prefill_2048", kind="attn", n_req=1, per_req=2048, rows_lo=2048, rows_hi=2048, page_rows=64,
             k_top=512, ratio=4, dtype="bf16"),
        # decode at ratio 128, every pooled row attended: ragged contexts up to 1M tokens (8192 rows)
        dict(name="attn_all_decode_24", kind="attn", n_req=24, per_req=1, rows_lo=1, rows_hi=8192, page_rows=32,
             k_top=0, ratio=128, dtype="bf16"),
        # one request alone with a very long pooled cache: the row axis has to be split
        dict(name="attn_all_decode_1", kind="attn", n_req=1, per_req=1, rows_lo=40001, rows_hi=40001, page_rows=64,
             k_top=0, ratio=128, dtype="f16"),
        # prefill chunks of three requests at ratio 128: every visible row, odd sizes
        dict(name="attn_all_prefill_3x211", kind="attn", n_req=3, per_req=211, rows_lo=200, rows_hi=1025,
             page_rows=16, k_top=0, ratio=128, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["plan", "append", "read", "attn", "attn", "attn", "attn"])
    ps = rng.choice([8, 16, 32, 64, 128, 256])
    dtype = rng.choice(["f16", "bf16"])
    if kind == "plan":
        hi = _log_int(rng, 1, 128)
        return dict(kind=kind, n_req=_log_int(rng, 1, 1500), new_lo=rng.choice([0, 1]), new_hi=hi,
                    seen_hi=_log_int(rng, 100, 65536), ratio=rng.choice([1, 3, 4, 7, 128]), page_rows=ps)
    if kind in ("append", "read"):
        return dict(kind=kind, n=_log_int(rng, 1, 50000), page_rows=ps, dtype=dtype)
    form = rng.choice(["decode", "decode", "prefill", "all_decode", "all_prefill"])
    if form == "decode":
        hi = _log_int(rng, 64, 65536)
        return dict(kind=kind, n_req=_log_int(rng, 1, 96), per_req=1, rows_lo=_log_int(rng, 1, hi), rows_hi=hi,
                    page_rows=ps, k_top=rng.choice([512, 512, 500, 64, 1024]), ratio=4, dtype=dtype)
    if form == "prefill":
        n_req = rng.choice([1, 1, 2, 5])
        hi = _log_int(rng, 32, 8192)
        return dict(kind=kind, n_req=n_req, per_req=max(2, _log_int(rng, 33, 2048) // n_req),
                    rows_lo=max(1, hi // 2), rows_hi=hi, page_rows=ps, k_top=rng.choice([512, 512, 333]), ratio=4,
                    dtype=dtype)
    if form == "all_decode":
        hi = _log_int(rng, 8, 16384)
        return dict(kind=kind, n_req=_log_int(rng, 1, 32), per_req=1, rows_lo=_log_int(rng, 1, hi), rows_hi=hi,
                    page_rows=ps, k_top=0, ratio=128, dtype=dtype)
    n_req = rng.choice([1, 2, 4])
    hi = _log_int(rng, 32, 1024)
    return dict(kind=kind, n_req=n_req, per_req=max(2, _log_int(rng, 16, 800) // n_req), rows_lo=max(1, hi // 3),
                rows_hi=hi, page_rows=ps, k_top=0, ratio=rng.choice([4, 128]), dtype=dtype)


def _attn_rows(case):
    """Rows a token attends to, about: for work()."""
    held = (case["rows_lo"] + case["rows_hi"]) / 2
    return min(case["k_top"], held) if case["k_top"] else held


def work(case):
    k = case["kind"]
    if k == "plan":
        tokens = case["n_req"] * (case["new_lo"] + case["new_hi"]) / 2
        pooled = tokens / case["ratio"]
        return {"bytes": 8 * tokens + 4 * pooled + 24 * case["n_req"] + 8 * pooled / case["page_rows"], "flops": 0}
    wide, packed = 2 * D, D // 2 + D // GROUP
    if k == "append":  # written, and the cache read back
        return {"bytes": case["n"] * (2 * wide + 2 * packed + 4), "flops": 0}
    if k == "read":
        return {"bytes": case["n"] * (wide + packed + 4), "flops": 0}
    T = case["n_req"] * case["per_req"]
    rows = _attn_rows(case)
    held = case["n_req"] * (case["rows_lo"] + case["rows_hi"]) / 2
    distinct = min(held, T * rows)  # each row of the cache that some token attends to is read once
    return {"bytes": T * HQ * D * 2 * 2 + distinct * packed + T * (4 * case["k_top"] + HQ * 4),
            "flops": 4 * T * HQ * D * rows}


# ----------------------------------------------------------------------------------------- inputs
def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed((seed * 1000003 + salt) % (2**62))


def _rows16(g, n, dtype):
    """Pooled rows: unit normal with a few loud channels and quiet rows."""
    x = torch.randn((n, D), generator=g, device="cuda")
    x[:, ::37] *= 4.0
    x *= torch.exp2(torch.randint(-3, 2, (n, 1), generator=g, device="cuda").float())
    return x.to(dtype)


def _pool(g, n_slots):
    codes = torch.empty((n_slots, D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n_slots, D // GROUP), dtype=torch.uint8, device="cuda")
    for a in range(0, n_slots, 1 << 17):
        n = min(1 << 17, n_slots - a)
        codes[a:a + n], scales[a:a + n] = _quantise(_rows16(g, n, torch.float16).float())
    return codes, scales


def prepare(case, seed):
    g = _gen(seed, 1)
    dev = "cuda"
    ps = case["page_rows"]
    if case["kind"] == "plan":
        B, ratio = case["n_req"], case["ratio"]
        seen = torch.randint(0, case["seen_hi"] + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        new = torch.randint(case["new_lo"], case["new_hi"] + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        rows = seen // ratio
        max_pages = ((case["seen_hi"] + case["new_hi"]) // ratio + ps) // ps
        n_pages = B * max_pages
        perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        held = (rows + ps - 1) // ps
        start = torch.cumsum(held, 0) - held
        col = torch.arange(max_pages, device=dev)
        at = (start[:, None] + col[None, :]).clamp_max(n_pages - 1)
        tables = torch.where(col[None, :] < held[:, None], perm[at], -1).to(torch.int32).contiguous()
        used = int(held.sum())
        want = int(((rows + (seen + new) // ratio - seen // ratio + ps - 1) // ps - held).sum())
        n_free = min(n_pages - used, max(1, want - want // 16))  # the last requests of a large step run short
        free = perm[used:].contiguous() if used < n_pages else perm[:1].contiguous()
        T_cap = B * case["new_hi"]
        R_cap = int(T_cap // ratio + B)
        return dict(case=case, seen=seen, new=new, rows=rows.to(torch.int32), tables=tables, free=free,
                    n_free=torch.tensor([n_free], dtype=torch.int32, device=dev), T_cap=T_cap, R_cap=R_cap)
    if case["kind"] in ("append", "read"):
        n = case["n"]
        n_slots = (n + n // 8 + ps) // ps * ps
        codes, scales = _pool(g, n_slots)
        slots = torch.randperm(n_slots, generator=g, device=dev)[:n].to(torch.int32)
        slots[torch.randint(0, n, (max(1, n // 64),), generator=g, device=dev)] = -1  # rows without a page
        s = dict(case=case, codes=codes, scales=scales, slots=slots)
        if case["kind"] == "append":
            s["x"] = _rows16(g, n, DTYPES[case["dtype"]])
            s["all"] = torch.arange(n_slots, dtype=torch.int32, device=dev)
        return s
    B, per, k_top, ratio = case["n_req"], case["per_req"], case["k_top"], case["ratio"]
    T = B * per
    u = torch.rand((B,), generator=g, device=dev)
    lo, hi = case["rows_lo"], case["rows_hi"]
    rows = torch.exp(math.log(lo) + u * (math.log(hi) - math.log(lo))).round().clamp(lo, hi).to(torch.int32)
    max_pages = (hi + ps - 1) // ps
    n_pages = B * max_pages + 1
    held = (rows + ps - 1) // ps
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)[:B * max_pages].reshape(B, max_pages)
    tables = torch.where(torch.arange(max_pages, device=dev)[None, :] < held[:, None], perm, -1).to(torch.int32)
    codes, scales = _pool(g, n_pages * ps)
    req = torch.arange(B, device=dev, dtype=torch.int32).repeat_interleave(per)
    # the last `per` positions of each request; the last one sees every held row
    positions = (rows[req.long()] * ratio - 1 - (per - 1 - torch.arange(per, device=dev).repeat(B))).to(torch.int32)
    q = torch.randn((T, HQ, D), generator=g, device=dev).to(DTYPES[case["dtype"]])
    s = dict(case=case, q=q, codes=codes, scales=scales, tables=tables.contiguous(), rows=rows, req=req,
             positions=positions, page_rows=ps, ratio=ratio, indices=None, counts=None)
    if k_top:
        n_vis = torch.minimum(rows[req.long()], ((positions + 1) // ratio).clamp_min(0)).to(torch.int32)
        # k_top distinct visible rows a token, ascending, -1 behind them: what the top-k emits
        width = max(k_top, int(n_vis.max()))
        idx = torch.empty((T, k_top), dtype=torch.int32, device=dev)
        step = max(1, (1 << 26) // width)
        for a in range(0, T, step):
            n = n_vis[a:a + step, None]
            key = torch.rand((n.shape[0], width), generator=g, device=dev)
            key = torch.where(torch.arange(width, device=dev)[None, :] < n, key, -1.0)
            v, i = key.topk(k_top, dim=1)
            i = torch.where(v >= 0, i, INT_MAX).sort(dim=1).values
            idx[a:a + step] = torch.where(i == INT_MAX, -1, i).to(torch.int32)
        s["indices"], s["counts"] = idx, torch.minimum(n_vis, torch.full_like(n_vis, k_top))
    return s


# ------------------------------------------------------------------------------------ plain forms
_HALF = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantise(x):
    """fp32 rows -> codes, scales.  Scaling by a power of two is exact, so the comparisons decide."""
    x = x.reshape(*x.shape[:-1], -1, GROUP)
    m, ex = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0.75, ex - 2, ex - 3).clamp(E_MIN, E_MAX)
    e = torch.where(m == 0, torch.full_like(e, E_MIN), e)
    y = torch.ldexp(x, -e[..., None])
    a = y.abs()
    # nearest, ties to the even code
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    c = c | (torch.signbit(y).to(torch.uint8) << 3)
    c = c.reshape(*c.shape[:-2], -1, 2)
    return (c[..., 0] | (c[..., 1] << 4)).contiguous(), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """codes [..., D/2], scales [..., D/32] -> fp32 values [..., D]."""
    one = torch.tensor(_HALF + tuple(-v for v in _HALF), device=codes.device)
    byte = torch.arange(256, device=codes.device)
    pair = torch.stack((one[byte & 15], one[byte >> 4]), -1)
    v = pair[codes.int()].reshape(*codes.shape[:-1], -1, GROUP)
    v = v * torch.exp2(scales.float() - 127.0)[..., None]
    return v.reshape(*codes.shape[:-1], -1)


def _plan_plain(s):
    c = s["case"]
    ratio, ps = c["ratio"], c["page_rows"]
    dev = s["seen"].device
    tables = s["tables"]
    max_pages = tables.shape[1]
    seen, new = s["seen"].long(), s["new"].long().clamp_min(0)
    r0 = s["rows"].long().clamp(0, max_pages * ps)
    done = (seen + new) // ratio - seen // ratio
    fits = torch.minimum(done, max_pages * ps - r0)
    held = (r0 + ps - 1) // ps
    need = (r0 + fits + ps - 1) // ps - held
    F = s["n_free"].long().clamp(0, s["free"].shape[0])
    first = torch.cumsum(need, 0) - need
    got = torch.minimum((F - first).clamp_min(0), need)
    placed = torch.minimum(fits, (held + got) * ps - r0)
    # new pages into the tables
    col = torch.arange(max_pages, device=dev)[None, :] - held[:, None]
    fresh = (col >= 0) & (col < got[:, None])
    at = (F - 1 - (first[:, None] + col)).clamp(0, s["free"].shape[0] - 1)
    tables.copy_(torch.where(fresh, s["free"][at], tables))
    # tokens
    T_cap, R_cap = s["T_cap"], s["R_cap"]
    ends = torch.cumsum(new, 0)
    t = torch.arange(T_cap, device=dev)
    b = torch.searchsorted(ends, t, right=True)
    live = b < new.shape[0]
    b = b.clamp_max(new.shape[0] - 1)
    positions = torch.where(live, seen[b] + t - (ends - new)[b], -1).to(torch.int32)
    req = torch.where(live, b, -1).to(torch.int32)
    # pooled rows
    ends = torch.cumsum(done, 0)
    j = torch.arange(R_cap, device=dev)
    b = torch.searchsorted(ends, j, right=True)
    live = b < new.shape[0]
    b = b.clamp_max(new.shape[0] - 1)
    i = j - (ends - done)[b]
    row = r0[b] + i
    page = tables[b, (row // ps).clamp(0, max_pages - 1)].long()
    slots = torch.where(live & (i < placed[b]) & (page >= 0), page * ps + row % ps, -1).to(torch.int32)
    taken = got.sum()
    totals = torch.stack((new.sum(), done.sum(), placed.sum(), taken)).to(torch.int32)
    return (positions, req, slots, tables, (seen + new).to(torch.int32), (r0 + placed).to(torch.int32),
            (F - taken).to(torch.int32), totals)


def _slots_of(s):
    """[T, n] slots of the rows each token attends to, and whether there is one."""
    r = s["req"].long()
    held = s["rows"].long()[r]
    if s["indices"] is None:
        n = torch.minimum(held, (s["positions"].long() + 1).clamp_min(0) // s["ratio"])
        row = torch.arange(s["tables"].shape[1] * s["page_rows"], device=r.device)[None, :].expand(r.shape[0], -1)
        live = row < n[:, None]
    else:
        row = s["indices"].long()
        live = (row >= 0) & (row < held[:, None])
        live &= torch.arange(row.shape[1], device=r.device)[None, :] < s["counts"].long()[:, None]
    row = torch.where(live, row, 0)
    page = s["tables"].long()[r[:, None], row // s["page_rows"]]
    live = live & (page >= 0)
    return torch.where(live, page * s["page_rows"] + row % s["page_rows"], 0), live


def _attn_plain(s):
    slot, live = _slots_of(s)
    kv = _values(s["codes"][slot], s["scales"][slot])                      # [T, n, D]
    x = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * (1.0 / math.sqrt(D))
    x = x.masked_fill(~live[:, None, :], float("-inf"))
    m = x.amax(-1, keepdim=True)
    m0 = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = torch.exp(x - m0)
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, kv) / torch.where(l > 0, l, torch.ones_like(l))
    return out.to(s["q"].dtype), (m0 + torch.log(l)).squeeze(-1)


def run(state):
    s = state
    kind = s["case"]["kind"]
    if not own:
        if kind == "plan":
            return _plan_plain(s)
        if kind == "read":
            ok = s["slots"] >= 0
            at = torch.where(ok, s["slots"], 0).long()
            v = _values(s["codes"][at], s["scales"][at])
            return torch.where(ok[:, None], v, 0.0).to(DTYPES[s["case"]["dtype"]])
        if kind == "append":
            c, e = _quantise(s["x"].float())
            ok = s["slots"] >= 0
            at = s["slots"][ok].long()
            s["codes"][at], s["scales"][at] = c[ok], e[ok]
            return _values(s["codes"], s["scales"]).to(s["x"].dtype)
        return _attn_plain(s)
    import deepseek_v4_sparse_gb300 as ds4x
    if kind == "plan":
        c = s["case"]
        positions, req, slots, seen, rows, n_free, totals = ds4x.page_plan(
            s["seen"], s["new"], s["rows"], s["tables"], s["free"], s["n_free"], c["ratio"], c["page_rows"],
            s["T_cap"], s["R_cap"])
        return positions, req, slots, s["tables"], seen, rows, n_free, totals
    if kind == "read":
        return ds4x.kv4_read(s["codes"], s["scales"], s["slots"], DTYPES[s["case"]["dtype"]])
    if kind == "append":
        ds4x.kv4_append(s["x"], s["slots"], s["codes"], s["scales"])
        return ds4x.kv4_read(s["codes"], s["scales"], s["all"], s["x"].dtype)
    return ds4x.kv4_attn(s["q"], s["codes"], s["scales"], s["tables"], s["rows"], s["page_rows"], req=s["req"],
                         positions=s["positions"], ratio=s["ratio"], indices=s["indices"], counts=s["counts"])


# ---------------------------------------------------------------------------------- 64-bit results
def _values64(codes, scales):
    """From the bits: sign, two exponent bits, one mantissa bit; the scale's exponent."""
    codes, scales = codes.to(torch.int64), scales.to(torch.int64)
    n = torch.stack((codes % 16, codes // 16), -1).reshape(*codes.shape[:-1], -1)
    ex, man = (n // 2) % 4, n % 2
    mag = torch.where(ex == 0, man.double() * 0.5, (1.0 + 0.5 * man.double()) * torch.exp2((ex - 1).double()))
    v = torch.where(n >= 8, -mag, mag)
    return v * torch.exp2((scales - 127).double()).repeat_interleave(GROUP, dim=-1)


def _append64(x):
    """Each value to the nearest of the sixteen, ties to the one with an even code; by distances."""
    x = x.double().cpu().numpy()
    grid = np.array(_HALF)
    out = np.empty_like(x)
    for a in range(0, x.shape[1], GROUP):
        blk = x[:, a:a + GROUP]
        top = np.abs(blk).max(axis=1)
        e = np.full(top.shape, E_MIN)
        for k in range(E_MIN, E_MAX):
            e = np.where(top > 6.0 * 2.0 ** k, k + 1, e)
        sc = 2.0 ** e.astype(np.float64)
        best, err = np.zeros_like(blk), np.full(blk.shape, np.inf)
        for code in (0, 2, 4, 6, 1, 3, 5, 7):  # even codes first: they keep a tie
            d = np.abs(np.abs(blk) - grid[code] * sc[:, None])
            best, err = np.where(d < err, grid[code] * sc[:, None], best), np.minimum(err, d)
        out[:, a:a + GROUP] = np.copysign(best, blk)
    return torch.from_numpy(out)


def exact(case, seed):
    if case["kind"] == "plan":
        return None
    s = prepare(case, seed)
    if case["kind"] == "read":
        v = _values64(s["codes"], s["scales"])
        z = torch.cat((v, torch.zeros_like(v[:1])))
        return z[torch.where(s["slots"] < 0, v.shape[0], s["slots"]).long()]
    if case["kind"] == "append":
        v = _values64(s["codes"], s["scales"])
        new = _append64(s["x"]).to(v.device)
        ok = s["slots"] >= 0
        v[s["slots"][ok].long()] = new[ok]
        return v
    q, T = s["q"].double(), s["q"].shape[0]
    out = torch.zeros((T, HQ, D), dtype=torch.float64, device=q.device)
    lse = torch.full((T, HQ), float("-inf"), dtype=torch.float64, device=q.device)
    req, rows, pos = s["req"].tolist(), s["rows"].tolist(), s["positions"].tolist()
    for t in range(T):
        b = req[t]
        if s["indices"] is None:
            take = torch.arange(max(0, min(rows[b], (pos[t] + 1) // s["ratio"])), device=q.device)
        else:
            take = s["indices"][t][:int(s["counts"][t])].long()
        if not len(take):
            continue
        at = s["tables"][b].long()[take // s["page_rows"]] * s["page_rows"] + take % s["page_rows"]
        kv = _values64(s["codes"][at], s["scales"][at])
        x = (q[t] @ kv.T) / math.sqrt(D)
        lse[t] = torch.logsumexp(x, 1)
        out[t] = torch.exp(x - lse[t][:, None]) @ kv
    return out, lse
