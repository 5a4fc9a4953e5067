"""Cases and plain forms of the operators of the paged 16-bit cache: the raw rows of many requests.

  rotate  rotate: the position rotation of queries on the way in, or of outputs on the way back (inverse)
  append  kv16_append: raw rows rotated by their positions and written to slots of the paged cache
  attn    kv16_attn: 64-head multi-query attention of decode tokens or chunks of new tokens over the cache

Rotation: the last `rot` values of a row are pairs (x0, x1), pair i of a row at position p becomes
(x0 cos a - x1 sin a, x1 cos a + x0 sin a) with a = p * inv_freq[i] (-a for the inverse).

Attention: row r of a request is the row of position r (of positions r * ratio .. r * ratio + ratio - 1).  A token
at position p of request b ends at row e = (p + 1) // ratio and sees the rows r of its request with
    max(first[t], e - window) <= r < min(rows[b], max(e, prefix[b]))
(no first, window or prefix: that bound is not there) whose page is in the table.  Its logits are
    x = scale q.kv_r,  cap * tanh(x / cap) with a cap,  less slopes[h] * |e - 1 - r| with slopes.
A sink adds exp(sinks[h]) to the normaliser of the softmax, and `other` joins the output and log-sum-exp of an
attention over other rows (the pooled ones) into the same softmax.
"""
import math

import torch

own = False

D, HQ = 512, 64
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------ cases
def _attn(name, n_req, per_req, rows_lo, rows_hi, page_rows, dtype, ratio=1, window=0, cap=0.0, slopes=False,
          sinks=False, other=False, doc=0, prefix=0):
    c = dict(kind="attn", n_req=n_req, per_req=per_req, rows_lo=rows_lo, rows_hi=rows_hi, page_rows=page_rows,
             dtype=dtype, ratio=ratio, window=window, cap=cap, slopes=slopes, sinks=sinks, other=other, doc=doc,
             prefix=prefix)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the queries of one decode step of 48 requests
        dict(name="rotate_decode_48", kind="rotate", n=48, heads=HQ, dim=D, rot=64, inverse=False, dtype="bf16"),
        # the outputs of a 2048-token prefill chunk, turned back
        dict(name="rotate_chunk_2048", kind="rotate", n=2048, heads=HQ, dim=D, rot=64, inverse=True, dtype="bf16"),
        # the raw rows of one decode step
        dict(name="append_decode_61", kind="append", n=61, rot=64, page_rows=64, dtype="bf16"),
        # the raw rows of long prompts of several requests
        dict(name="append_prefill_50001", kind="append", n=50001, rot=64, page_rows=64, dtype="f16"),
        # the first decode steps of one short request: latency
        _attn("attn_decode_1_short", 1, 1, 77, 77, 64, "bf16"),
        # one request alone with a long cache, every row attended: the row axis has to be split
        _attn("attn_decode_1_long", 1, 1, 120001, 120001, 64, "bf16"),
        # a decode batch of ragged contexts with capped logits
        _attn("attn_decode_61", 61, 1, 5, 32768, 32, "f16", cap=30.0),
        # a large decode batch over its last 128 rows, joined with what the pooled rows gave
        _attn("attn_window_256", 256, 1, 40, 9000, 16, "bf16", window=128, sinks=True, other=True),
        # a 2048-token prefill chunk over its last 128 rows each, joined with what the pooled rows gave
        _attn("attn_window_chunk_2048", 1, 2048, 6001, 6001, 64, "bf16", window=128, sinks=True, other=True),
        # a chunk of new tokens late in a long prompt, every row attended
        _attn("attn_chunk_512", 1, 512, 8192, 8192, 64, "bf16"),
        # chunks of four requests with a bias that grows with the distance, odd sizes
        _attn("attn_chunk_bias_4x101", 4, 101, 300, 2500, 16, "f16", cap=50.0, slopes=True),
        # whole prompts of packed documents, the first of which is a prefix that sees itself both ways
        _attn("attn_docs_2x1021", 2, 1021, 1021, 1021, 32, "f16", doc=389, prefix=150),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rotate", "append", "attn", "attn", "attn", "attn"])
    dtype = rng.choice(["f16", "bf16"])
    if kind == "rotate":
        heads, dim = rng.choice([(64, 512), (64, 512), (1, 512), (64, 128), (32, 128), (1, 128)])
        rot = rng.choice([r for r in (32, 64, 64, 128, 512) if r <= dim])
        return dict(kind=kind, n=_log_int(rng, 1, 2048), heads=heads, dim=dim, rot=rot,
                    inverse=rng.choice([False, True]), dtype=dtype)
    ps = rng.choice([8, 16, 32, 64, 128, 256])
    if kind == "append":
        return dict(kind=kind, n=_log_int(rng, 1, 50000), rot=rng.choice([0, 32, 64, 64, 128, 512]), page_rows=ps,
                    dtype=dtype)
    opts = dict(cap=rng.choice([0.0, 0.0, 20.0, 50.0]), slopes=rng.random() < 0.25, sinks=rng.random() < 0.35,
                other=rng.random() < 0.35)
    form = rng.choice(["decode", "decode", "decode_window", "window", "chunk", "docs"])
    if form == "decode":
        n_req = _log_int(rng, 1, 96)
        hi = _log_int(rng, 8, min(120000, 380000 // n_req))
        return _attn(None, n_req, 1, _log_int(rng, 1, hi), hi, ps, dtype, ratio=rng.choice([1, 1, 4, 128]), **opts)
    if form == "decode_window":
        hi = _log_int(rng, 8, 9000)
        return _attn(None, _log_int(rng, 1, 256), 1, _log_int(rng, 1, hi), hi, ps, dtype,
                     window=rng.choice([128, 128, 1, 77, 512, 1024]), **opts)
    n_req = rng.choice([1, 1, 2, 5])
    if form == "window":
        per = max(2, _log_int(rng, 33, 2048) // n_req)
        hi = per + _log_int(rng, 1, 6000)
        return _attn(None, n_req, per, per, hi, ps, dtype, window=rng.choice([128, 128, 64, 200]), **opts)
    if form == "chunk":
        per = max(2, _log_int(rng, 8, 512) // n_req)
        hi = per + _log_int(rng, 1, 7000)
        return _attn(None, n_req, per, max(per, hi // 3), hi, ps, dtype, **opts)
    per = max(2, _log_int(rng, 50, 1800) // n_req)
    return _attn(None, n_req, per, per, per, ps, dtype, doc=rng.choice([0, _log_int(rng, 5, 700)]),
                 prefix=rng.choice([0, _log_int(rng, 2, 300)]), **opts)


def _rows_held(c):
    """Rows of each request, ascending: spread over the logarithm, the same for every seed."""
    B, lo, hi = c["n_req"], c["rows_lo"], c["rows_hi"]
    return [max(lo, min(hi, round(lo * (hi / lo) ** ((b + 0.5) / B)))) for b in range(B)]


def _span(c, held, p):
    """First and last (exclusive) row that a token at position p sees of a request with `held` rows."""
    e = (p + 1) // c["ratio"]
    lo = max(0, e - c["window"]) if c["window"] else 0
    if c["doc"]:
        lo = max(lo, p // c["doc"] * c["doc"])
    return lo, max(lo, min(held, max(e, min(c["prefix"], held))))


def _first_position(c, held):
    return held * c["ratio"] - c["per_req"]


def work(case):
    k = case["kind"]
    if k == "rotate":
        n = case["n"] * case["heads"] * case["dim"]
        return {"bytes": 4 * n + 4 * case["n"], "flops": 0}
    if k == "append":
        return {"bytes": case["n"] * (4 * D + 8), "flops": 0}
    pairs = distinct = 0
    for held in _rows_held(case):
        p0 = _first_position(case, held)
        spans = [_span(case, held, p0 + i) for i in range(case["per_req"])]
        pairs += sum(b - a for a, b in spans)
        seen = [s for s in spans if s[1] > s[0]]
        if seen:
            distinct += max(b for _, b in seen) - min(a for a, _ in seen)
    T = case["n_req"] * case["per_req"]
    q = T * HQ * D * 2
    return {"bytes": (3 if case["other"] else 2) * q + distinct * D * 2 + T * HQ * 4 * (2 if case["other"] else 1),
            "flops": 4 * HQ * D * pairs}


# ----------------------------------------------------------------------------------------- inputs
def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed((seed * 1000003 + salt) % (2**62))


def _rows16(g, n, dtype):
    """Rows: unit normal with a few loud channels and quiet rows."""
    x = torch.randn((n, D), generator=g, device="cuda")
    x[:, ::37] *= 4.0
    x *= torch.exp2(torch.randint(-3, 2, (n, 1), generator=g, device="cuda").float())
    return x.to(dtype)


def _inv_freq(rot):
    i = torch.arange(0, rot, 2, dtype=torch.float64, device="cuda")
    return torch.pow(10000.0, -i / rot)


def prepare(case, seed):
    g = _gen(seed, 2)
    dev = "cuda"
    dt = DTYPES[case["dtype"]]
    if case["kind"] == "rotate":
        shape = (case["n"], case["heads"], case["dim"])
        x = torch.randn(shape, generator=g, device=dev).to(dt)
        # consecutive positions somewhere in a long context, and a few tokens of other requests
        p0 = int(torch.randint(0, 1 << 20, (1,), generator=g, device=dev))
        pos = p0 + torch.arange(case["n"], device=dev, dtype=torch.int32)
        pos[::5] = torch.randint(0, 1 << 20, (len(pos[::5]),), generator=g, device=dev, dtype=torch.int32)
        return dict(case=case, x=x, positions=pos, inv_freq=_inv_freq(case["rot"]))
    ps = case["page_rows"]
    if case["kind"] == "append":
        n = case["n"]
        n_slots = (n + n // 8 + ps) // ps * ps
        pool = torch.zeros((n_slots, D), dtype=dt, device=dev)
        slots = torch.randperm(n_slots, generator=g, device=dev)[:n].to(torch.int32)
        slots[torch.randint(0, n, (n // 50,), generator=g, device=dev)] = -1  # rows without a page
        pos = torch.randint(0, 1 << 20, (n,), generator=g, device=dev, dtype=torch.int32)
        return dict(case=case, x=_rows16(g, n, dt), slots=slots, pool=pool, positions=pos if case["rot"] else None,
                    inv_freq=_inv_freq(case["rot"]) if case["rot"] else None)
    B, per, ratio, window = case["n_req"], case["per_req"], case["ratio"], case["window"]
    T = B * per
    host_rows = _rows_held(case)
    order = torch.randperm(B, generator=g, device=dev).tolist()
    host_rows = [host_rows[i] for i in order]
    max_pages = (max(host_rows) + ps - 1) // ps
    # pages wholly before what the step's tokens see have gone back to the free list
    keep = []
    for held in host_rows:
        p0 = _first_position(case, held)
        lo = min(_span(case, held, p0 + i)[0] for i in range(per)) if window else 0
        keep.append((lo // ps, (held + ps - 1) // ps))
    n_pages = sum(b - a for a, b in keep) + 1
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    tables = torch.full((B, max_pages), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, (a, z) in enumerate(keep):
        tables[b, a:z] = perm[at:at + z - a]
        at += z - a
    pool = torch.empty((n_pages * ps, D), dtype=dt, device=dev)
    for a in range(0, n_pages * ps, 1 << 17):
        z = min(n_pages * ps, a + (1 << 17))
        pool[a:z] = _rows16(g, z - a, dt)
    rows = torch.tensor(host_rows, dtype=torch.int32, device=dev)
    req = torch.arange(B, device=dev, dtype=torch.int32).repeat_interleave(per)
    positions = (rows[req.long()] * ratio - per + torch.arange(per, device=dev, dtype=torch.int32).repeat(B))
    s = dict(case=case, q=torch.randn((T, HQ, D), generator=g, device=dev).to(dt), pool=pool, tables=tables, rows=rows,
             req=req, positions=positions.to(torch.int32), page_rows=ps, ratio=ratio, window=window, cap=case["cap"],
             first=None, prefix=None, slopes=None, sinks=None, other=None, host_rows=host_rows)
    if case["doc"]:
        s["first"] = (s["positions"] // case["doc"] * case["doc"]).to(torch.int32)
    if case["prefix"]:
        s["prefix"] = torch.minimum(rows, torch.full_like(rows, case["prefix"]))
    if case["slopes"]:
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, HQ + 1, device=dev).float() / HQ)
    if case["sinks"]:
        s["sinks"] = torch.randn((HQ,), generator=g, device=dev) * 2.0
    if case["other"]:
        o = torch.randn((T, HQ, D), generator=g, device=dev).mul_(0.3).to(dt)
        l = 4.0 + torch.randn((T, HQ), generator=g, device=dev)
        none = torch.arange(T, device=dev) % 97 == 96  # tokens that selected no pooled row
        o[none] = 0
        l[none] = float("-inf")
        s["other"] = (o, l)
    return s


# ------------------------------------------------------------------------------------ plain forms
def _rotated(x, positions, inv_freq, inverse):
    """fp32 x [..., dim], positions broadcast over all but the last axis; angles in 64 bits."""
    rot = 2 * inv_freq.shape[0]
    a = positions.double()[..., None] * inv_freq
    c, s = torch.cos(a).float(), torch.sin(a).float()
    if inverse:
        s = -s
    tail = x[..., x.shape[-1] - rot:]
    x0, x1 = tail[..., 0::2], tail[..., 1::2]
    turned = torch.stack((x0 * c - x1 * s, x1 * c + x0 * s), -1).flatten(-2)
    return torch.cat((x[..., :x.shape[-1] - rot], turned), -1)


def _softmax_plain(s, q, kv, r, live, e, t):
    """q [n, HQ, D] of the tokens t over kv [n or 1, rows, D]; r (row numbers) and live [n, rows]; e [n]."""
    c = s["case"]
    x = torch.matmul(q.float(), kv.transpose(1, 2)) * (1.0 / math.sqrt(D))
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    if s["slopes"] is not None:
        x = x - s["slopes"][:, None] * (e[:, None] - 1 - r).abs().float()[:, None, :]
    x = x.masked_fill(~live[:, None, :], float("-inf"))
    m = x.amax(-1)
    if s["sinks"] is not None:
        m = torch.maximum(m, s["sinks"])
    if s["other"] is not None:
        m = torch.maximum(m, s["other"][1][t])
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    x = torch.exp(x - m[..., None])
    l = x.sum(-1)
    o = torch.matmul(x, kv)
    if s["sinks"] is not None:
        l = l + torch.exp(s["sinks"] - m)
    if s["other"] is not None:
        w = torch.exp(s["other"][1][t] - m)
        l = l + w
        o = o + w[..., None] * s["other"][0][t].float()
    return o / torch.where(l > 0, l, torch.ones_like(l))[..., None], m + torch.log(l)


def _attn_plain(s):
    c = s["case"]
    per, ps, dev = c["per_req"], c["page_rows"], s["q"].device
    T = s["q"].shape[0]
    out = torch.empty_like(s["q"])
    lse = torch.empty((T, HQ), dtype=torch.float32, device=dev)
    held, req = s["rows"].long()[s["req"].long()], s["req"].long()
    e = (s["positions"].long() + 1) // c["ratio"]
    lo = (e - c["window"] if c["window"] else torch.zeros_like(e)).clamp_min(0)
    if s["first"] is not None:
        lo = torch.maximum(lo, s["first"].long())
    hi = torch.minimum(held, e if s["prefix"] is None else torch.maximum(e, s["prefix"].long()[req]))
    if per == 1:  # tokens of different requests: each with its own rows, padded to the longest list
        width = max(1, min(c["window"] or c["rows_hi"], c["rows_hi"]))
        groups = [(a, min(T, a + max(1, (1 << 22) // width)), None) for a in
                  range(0, T, max(1, (1 << 22) // width))]
    else:  # tokens of one request share its rows
        groups = []
        for b, n in enumerate(s["host_rows"]):
            base = _span(c, n, _first_position(c, n))[0] if c["window"] else 0
            step = max(1, (1 << 29) // (HQ * max(1, n - base)))
            groups += [(b * per + i, b * per + min(per, i + step), (base, n)) for i in range(0, per, step)]
    for a, z, span in groups:
        t = slice(a, z)
        if span is None:
            r = lo[t, None] + torch.arange(width, device=dev)
            col = (r // ps).clamp_max(s["tables"].shape[1] - 1)
            page = s["tables"].long()[req[t, None], col]
        else:
            r = torch.arange(span[0], span[1], device=dev)[None, :]
            page = s["tables"][a // per].long()[r // ps]
        kv = s["pool"][page.clamp_min(0) * ps + r % ps].float()
        live = (r >= lo[t, None]) & (r < hi[t, None]) & (page >= 0)
        o, lse[t] = _softmax_plain(s, s["q"][t], kv, r, live, e[t], t)
        out[t] = o.to(out.dtype)
    return out, lse


def run(state):
    s = state
    kind = s["case"]["kind"]
    if not own:
        if kind == "rotate":
            x = s["x"].float()
            return _rotated(x, s["positions"][:, None], s["inv_freq"], s["case"]["inverse"]).to(s["x"].dtype)
        if kind == "append":
            x = s["x"].float()
            if s["inv_freq"] is not None:
                x = _rotated(x, s["positions"], s["inv_freq"], False)
            ok = s["slots"] >= 0
            s["pool"][s["slots"][ok].long()] = x[ok].to(s["pool"].dtype)
            return s["pool"]
        return _attn_plain(s)
    import deepseek_v4_sparse_gb300 as ds4x
    if kind == "rotate":
        return ds4x.rotate(s["x"], s["positions"], s["inv_freq"], inverse=s["case"]["inverse"])
    if kind == "append":
        ds4x.kv16_append(s["x"], s["slots"], s["pool"], positions=s["positions"], inv_freq=s["inv_freq"])
        return s["pool"]
    return ds4x.kv16_attn(s["q"], s["pool"], s["tables"], s["rows"], s["page_rows"], req=s["req"],
                          positions=s["positions"], ratio=s["ratio"], window=s["window"], first=s["first"],
                          prefix=s["prefix"], cap=s["cap"], slopes=s["slopes"], sinks=s["sinks"], other=s["other"])


# ---------------------------------------------------------------------------------- 64-bit results
def _turn64(x, positions, inv_freq, inverse):
    """x [n, heads, dim]: the pairs as complex numbers, turned by a unit number."""
    z = x.double().clone()
    rot = 2 * inv_freq.numel()
    pairs = torch.view_as_complex(z[:, :, z.shape[2] - rot:].reshape(*z.shape[:2], -1, 2).contiguous())
    angle = torch.outer(positions.double(), inv_freq)
    unit = torch.polar(torch.ones_like(angle), -angle if inverse else angle)
    z[:, :, z.shape[2] - rot:] = torch.view_as_real(pairs * unit[:, None, :]).reshape(*z.shape[:2], rot)
    return z


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "rotate":
        return _turn64(s["x"], s["positions"], s["inv_freq"], case["inverse"])
    if case["kind"] == "append":
        x = s["x"][:, None, :]
        x = (_turn64(x, s["positions"], s["inv_freq"], False) if case["rot"] else x.double())[:, 0]
        pool = torch.cat((s["pool"].double(), torch.zeros((1, D), dtype=torch.float64, device=x.device)))
        pool[torch.where(s["slots"] < 0, pool.shape[0] - 1, s["slots"]).long()] = x
        return pool[:-1]
    T = s["q"].shape[0]
    dev = s["q"].device
    out = torch.zeros((T, HQ, D), dtype=torch.float64, device=dev)
    lse = torch.full((T, HQ), float("-inf"), dtype=torch.float64, device=dev)
    ps, pos, req = case["page_rows"], s["positions"].tolist(), s["req"].tolist()
    slopes, sinks = ((None if s[k] is None else s[k].double()) for k in ("slopes", "sinks"))
    caches = {}
    for t in range(T):
        held = s["host_rows"][req[t]]
        lo, hi = _span(case, held, pos[t])
        if req[t] not in caches:
            caches.clear()
            low = lo if case["window"] else 0
            r = torch.arange(low, held, device=dev)
            at = s["tables"][req[t]].long()[r // ps] * ps + r % ps
            caches[req[t]] = (low, s["pool"][at].double())
        low, kv = caches[req[t]]
        kv = kv[lo - low:hi - low]
        x = s["q"][t].double() @ kv.T * D ** -0.5
        if case["cap"]:
            x = torch.tanh(x / case["cap"]) * case["cap"]
        if slopes is not None:
            away = (torch.arange(lo, hi, device=dev) - ((pos[t] + 1) // case["ratio"] - 1)).abs().double()
            x = x - torch.outer(slopes, away)
        terms = [x]
        if sinks is not None:
            terms.append(sinks[:, None])
        if s["other"] is not None:
            terms.append(s["other"][1][t].double()[:, None])
        total = torch.logsumexp(torch.cat(terms, 1), 1)
        lse[t] = total
        gone = torch.isneginf(total)[:, None]
        o = torch.where(gone, 0.0, torch.exp(x - total[:, None])) @ kv
        if s["other"] is not None:
            o = o + torch.where(gone, 0.0, torch.exp(terms[-1] - total[:, None])) * s["other"][0][t].double()
        out[t] = o
    return out, lse
