"""The paged 16-bit cache on the GPU against its plain implementation in 64 bits (oracle/kv16.py)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import deepseek_v4_sparse_gb300 as ds4x
from oracle import kv4, kv16

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
I32 = torch.int32
SCALE = 512 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deepseek_v4_sparse_gb300 import build
    build.build()
    ds4x.load()
    yield
    torch.cuda.synchronize()
    assert ds4x.device_status() == ds4x.OK


def gpu(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def i32(a):
    return gpu(np.asarray(a, dtype=np.int32))


def frequencies(rot, base=10000.0):
    return base ** (-np.arange(0, rot, 2) / rot)


# -------------------------------------------------------------------------------------- rotation
def turn_tolerance(y, x, positions, f, dtype):
    """Half a step of the type for the one rounding (fp16 below its normal range: 2^-25), and the pair's length
    times what the angle may be off: |p| (f + 1) 2^-51 + 2^-22 of the call, |p| f 2^-53 of the 64-bit angle here,
    and 2^-22 for cos, sin and the two products in fp32."""
    half = torch.finfo(DT[dtype]).eps / 2
    tol = half * 1.001 * np.abs(y) + (2.0 ** -25 if dtype == "f16" else 0.0)
    start = y.shape[-1] - 2 * len(f)
    length = np.hypot(x[..., start::2], x[..., start + 1::2])
    p = np.abs(np.asarray(positions, dtype=np.float64)).reshape((-1,) + (1,) * (y.ndim - 1))
    off = length * (p * (f + 1) * 2.0 ** -50.5 + 2.0 ** -21)
    tol[..., start:] += np.repeat(off, 2, axis=-1)
    return tol


POSITIONS = [0, 1, -1, 77, 1 << 20, 999999, 2 ** 31 - 1, -2 ** 31, 12345678]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,H,D,rot", [(1, 64, 512, 64), (9, 64, 512, 64), (5, 3, 128, 128), (9, 1, 512, 512),
                                       (4, 64, 72, 10), (2, 1, 8, 2), (3, 5, 64, 6), (7, 33, 4096, 4096)])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotate(T, H, D, rot, dtype, inverse):
    rng = np.random.default_rng(T * 7 + rot)
    x = torch.from_numpy(rng.standard_normal((T, H, D)) * 3).to(DT[dtype])
    pos, f = np.array(POSITIONS[:T]), frequencies(rot)
    args = i32(pos), gpu(f)
    ref = kv16.rotate(x.double().numpy(), pos, f, inverse)
    tol = turn_tolerance(ref, x.double().numpy(), pos, f, dtype)
    dx = x.cuda()
    y = ds4x.rotate(dx, *args, inverse=inverse)
    assert torch.equal(dx.cpu(), x)
    got = y.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= tol), (np.abs(got - ref) / tol).max()
    assert torch.equal(y[..., :D - rot].cpu(), x[..., :D - rot])
    assert ds4x.rotate(dx, *args, inverse=inverse, out=dx) is dx and torch.equal(dx, y)   # in place
    if H == 1:
        assert torch.equal(ds4x.rotate(x[:, 0].contiguous().cuda(), *args, inverse=inverse), y[:, 0])


def test_rotate_back_and_odd_values():
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((6, 64, 512))).bfloat16()
    x[0, 0, 0], x[1, 1, 447], x[2, 2, 100] = float("nan"), float("inf"), float("-inf")   # not rotated
    x[3, 3, 448], x[4, 4, 511] = float("nan"), float("inf")
    pos, f = i32([5, 1 << 20, 77, 3, 0, -9]), gpu(frequencies(64))
    y = ds4x.rotate(x.cuda(), pos, f)
    z = ds4x.rotate(y, pos, f, inverse=True).cpu()
    assert torch.equal(z[..., :448].view(torch.int16), x[..., :448].view(torch.int16))
    odd = ~torch.isfinite(x[..., 448:])
    odd |= odd.reshape(6, 64, 32, 2).flip(-1).reshape(6, 64, 64)                         # and their partners
    got, want = z[..., 448:].double()[~odd], x[..., 448:].double()[~odd]
    # two roundings of numbers no longer than their pair, and the pair's length 2^-20 for two inexact angles
    length = x[..., 448:].double().reshape(6, 64, 32, 2).norm(dim=-1, keepdim=True).expand(6, 64, 32, 2)
    tol = 2.0 * 2.0 ** -8 * length.reshape(6, 64, 64)[~odd] * 1.01
    assert torch.all((got - want).abs() <= tol)
    assert not torch.isfinite(y.cpu()[..., 448:][odd]).any()


def test_rotate_more_tokens_than_a_grid_axis():
    T = 70001
    x = torch.randn((T, 8), device="cuda").half()
    pos = torch.arange(T, dtype=I32, device="cuda")
    f = gpu([0.7, 1e-4])
    y = ds4x.rotate(x, pos, f)
    pick = torch.tensor([0, 1, 65534, 65535, 65536, 70000])
    ref = kv16.rotate(x[pick].double().cpu().numpy(), pick.numpy(), f.cpu().numpy())
    tol = turn_tolerance(ref, x[pick].double().cpu().numpy(), pick.numpy(), f.cpu().numpy(), "f16")
    assert np.all(np.abs(y[pick].double().cpu().numpy() - ref) <= tol)
    assert ds4x.rotate(x[:0], pos[:0], f).shape == (0, 8)


# ---------------------------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n,rot", [(0, 64), (1, 64), (7, 64), (61, 64), (300, 0), (300, 512), (1301, 2), (5000, 10),
                                   (20011, 64)])
def test_append(n, rot, dtype):
    rng = np.random.default_rng(n + rot)
    x = torch.from_numpy(rng.standard_normal((n, 512)) * 2).to(DT[dtype])
    n_slots = n + 11
    slots = rng.permutation(n_slots)[:n].astype(np.int32)
    if n >= 7:
        slots[::5] = -1
        slots[1], slots[3] = n_slots, 2 ** 31 - 1
        x[2, 17] = float("nan")
    pos = rng.integers(0, 1 << 20, n).astype(np.int32)
    before = torch.from_numpy(rng.standard_normal((n_slots, 512))).to(DT[dtype])
    pool, f = before.cuda(), frequencies(rot) if rot else None
    ds4x.kv16_append(x.cuda(), i32(slots), pool, **(dict(positions=i32(pos), inv_freq=gpu(f)) if rot else {}))
    got = pool.cpu()
    ok = (slots >= 0) & (slots < n_slots)
    kept = np.setdiff1d(np.arange(n_slots), slots)
    assert torch.equal(got[kept], before[kept])
    at, xs = slots[ok], x[torch.from_numpy(ok)]
    assert torch.equal(got[at][:, :512 - rot].view(torch.int16), xs[:, :512 - rot].view(torch.int16))
    if rot and ok.any():
        xn = torch.nan_to_num(xs).double().numpy()
        ref = kv16.rotate(xn, pos[ok], f)
        tol = turn_tolerance(ref, xn, pos[ok], f, dtype)[:, 512 - rot:]
        g, w = got[at].double().numpy()[:, 512 - rot:], ref[:, 512 - rot:]
        sure = torch.isfinite(xs).numpy()[:, 512 - rot:].reshape(len(at), -1, 2).all(-1).repeat(2, axis=-1)
        assert np.all((np.abs(g - w) <= tol) | ~sure)


# ------------------------------------------------------------------------------------- attention
class Pool:
    """A pool of random rows; whatever no request holds is NaN, and so is every page of a request before `gone`
    rows of it, which the table no longer names."""

    def __init__(self, rng, rows, ps, dtype, gone=None, size=1.0):
        self.rows, self.ps = np.asarray(rows, dtype=np.int32), ps
        B = len(self.rows)
        held = -(-self.rows // ps)
        skip = [0] * B if gone is None else [g // ps for g in gone]
        self.max_pages = max(1, int(held.max(initial=0)))
        n_pages = int(held.sum()) + 3
        self.n_slots = n_pages * ps
        pages = rng.permutation(n_pages)
        self.tables = np.full((B, self.max_pages), -1, dtype=np.int32)
        pool = torch.full((self.n_slots, 512), float("nan"), dtype=DT[dtype])
        k = 0
        for b in range(B):
            for pg in range(skip[b], held[b]):
                self.tables[b, pg] = pages[k]
                k += 1
                n = min(ps, self.rows[b] - pg * ps)
                x = rng.standard_normal((n, 512)) * size * np.exp2(rng.integers(-3, 2, (n, 1)).astype(float))
                at = self.tables[b, pg] * ps
                pool[at:at + n] = torch.from_numpy(x).to(DT[dtype])
        self.dev = pool.cuda(), i32(self.tables), i32(self.rows)

    def values(self):
        return self.dev[0].double().cpu().numpy()


def tolerance(x, kv, w, out, dtype, cap):
    """How far out [H, 512] and lse [H] of one token may be: logits x [H, n] of the rows kv [n, 512] (the other
    attention's output and the sink among them, if any) with normalised weights w [H, n]; `x` comes with ex [H],
    the bound on what a logit may be off.

    A weight moves by 2 ex + 2^-20 (2^x and its argument, whose size counts: 2^-23 |x|) relative, and is rounded
    to `dtype` once, half a step u, in numerator and normaliser alike: a normalised weight moves by at most
    eta = 2 (u + 2 ex'), and |out - ref| <= eta sum_j w_j |kv_j - ref|.  The largest weight of a head is at least
    one before the sum, so those below fp16's normal range are off by 2^-25 each at most against it.
    The output is rounded once: half a step, 2^-25 below fp16's normal range."""
    logit, ex = x
    u = torch.finfo(DT[dtype]).eps / 2
    size = np.where(np.isfinite(logit), np.abs(logit), 0).max(axis=1, initial=0.0)
    # capped, a logit is off by 2^-21 of the cap (2 / (e^2y + 1), each of its three steps by 2^-22 at most) up to a cap of
    # 256.  Above, by as much where it is over 0.24 of the cap, that is by 2^-18.9 of itself, and by less elsewhere
    ex = ex + 2.0 ** -20 + (2.0 ** -18.5 if cap > 256 else 2.0 ** -22) * size + (cap * 2.0 ** -20 if cap <= 256 else 0.0)
    eta = 2 * (u + 2 * ex)
    spread = np.stack([w[h] @ np.abs(kv[h] - out[h][None, :]) for h in range(w.shape[0])])
    tiny = kv.shape[1] * 2.0 ** -25 * np.abs(kv).max(initial=0.0) * (dtype == "f16")
    return (eta[:, None] * spread + tiny + u * 1.01 * np.abs(out) + 2.0 ** -25, 2 * ex)


def check_attn(q, pool, got, lse, dtype, scale, opts, lists, tokens=None):
    vals = pool.values()
    T = q.shape[0]
    qd, g, gl = q.double().cpu().numpy(), got.double().cpu().numpy(), lse.double().cpu().numpy()
    host = {k: v for k, v in opts.items()}
    if "other" in host:
        host["other"] = tuple(t.double().cpu().numpy() for t in host["other"])
    for t in range(T) if tokens is None else tokens:
        one = {k: (v[t:t + 1] if k in ("req", "positions", "first") and v is not None else v) for k, v in lists.items()}
        if one.get("req") is None:
            one["req"] = [t]
        if "other" in host:
            one_host = dict(host, other=(host["other"][0][t:t + 1], host["other"][1][t:t + 1]))
        else:
            one_host = host
        tabs = dict(tables=pool.tables, rows=pool.rows, page_rows=pool.ps)
        ref, rlse = kv16.attn(qd[t:t + 1], vals, scale, **one_host, **tabs, **one)
        ref, rlse = ref[0], rlse[0]
        e, see, at = kv16.seen_rows(0, n_slots=pool.n_slots, **tabs, **one)
        none = np.isneginf(rlse)
        assert np.all(np.isneginf(gl[t][none])) and np.all(g[t][none] == 0), t
        if none.all():
            continue
        kv = vals[at] if at else np.zeros((0, 512))
        x = kv16.logits(qd[t], kv, see, e, scale, opts.get("cap", 0.0), opts.get("slopes")) if at else np.zeros((64, 0))
        # 512 exact products summed in fp32 by a truncating adder, 64 steps of at most 2^-23 of the magnitudes
        ex = 64 * 2.0 ** -23 * scale * (np.abs(qd[t]) @ np.abs(kv).T).max(axis=1, initial=0.0)
        kvh = np.broadcast_to(kv, (64,) + kv.shape)
        if "sinks" in opts:
            x = np.concatenate([x, np.asarray(opts["sinks"])[:, None]], 1)
            kvh = np.concatenate([kvh, np.zeros((64, 1, 512))], 1)
        if "other" in opts:
            ol = one_host["other"][1][0]
            x = np.concatenate([x, ol[:, None]], 1)
            kvh = np.concatenate([kvh, np.where(np.isneginf(ol)[:, None], 0.0, one_host["other"][0][0])[:, None, :]], 1)
        with np.errstate(invalid="ignore"):
            w = np.where(none[:, None], 0.0, np.exp(x - rlse[:, None]))
        tol, ltol = tolerance((x, ex), kvh, w, ref, dtype, opts.get("cap", 0.0))
        assert np.all(np.isfinite(g[t][~none])), t
        worst = (np.abs(g[t] - ref) / tol).max()
        assert worst <= 1, (t, len(at), worst)
        assert np.all(np.abs(gl[t][~none] - rlse[~none]) <= ltol[~none]), t


def queries(rng, T, dtype, size=1.0):
    return torch.from_numpy(rng.standard_normal((T, 64, 512)) * size).to(DT[dtype]).cuda()


def on_gpu(opts, lists):
    kw = {k: (v if k in ("ratio", "window") or v is None else i32(v)) for k, v in lists.items()}
    for k, v in opts.items():
        kw[k] = v if k in ("cap", "other") else gpu(np.asarray(v, dtype=np.float32))
    return kw


def run_attn(q, pool, opts, lists, **kw):
    return ds4x.kv16_attn(q, *pool.dev, pool.ps, **on_gpu(opts, lists), **kw)


def options(rng, T, dtype, cap=False, slopes=False, sinks=False, other=False):
    o = {}
    if cap:
        o["cap"] = 1.5
    if slopes:
        o["slopes"] = np.float32(np.exp2(-rng.uniform(0, 9, 64)))
    if sinks:
        o["sinks"] = np.float32(rng.standard_normal(64) * 3)
        o["sinks"][5] = -np.inf
    if other:
        lse = torch.from_numpy(rng.standard_normal((T, 64)) * 2 + 2).float()
        out = torch.from_numpy(rng.standard_normal((T, 64, 512))).to(DT[dtype])
        lse[::3] = float("-inf")               # tokens of which the other attention saw nothing:
        out[::3] = float("nan")                # what it wrote for them is not looked at
        o["other"] = out.cuda(), lse.cuda()
    return o


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,ps", [
    ([1], 64), ([2], 1), ([15], 8), ([16], 16), ([17], 16), ([64], 64), ([127], 32), ([128], 128), ([129], 4),
    ([255], 64), ([700], 64), ([300, 1, 65, 0, 128, 129, 31], 16), ([2000, 1500], 256), ([5000], 2),
])
def test_attn_all_rows(rows, ps, dtype):
    """A token a request, every row held; no positions, then the positions that mean the same."""
    rng = np.random.default_rng(sum(rows) + ps)
    pool = Pool(rng, rows, ps, dtype)
    q = queries(rng, len(rows), dtype)
    out, lse = run_attn(q, pool, {}, {})
    check_attn(q, pool, out, lse, dtype, SCALE, {}, {})
    lists = dict(req=np.arange(len(rows)), positions=np.asarray(rows) - 1)
    out2, lse2 = run_attn(q, pool, {}, lists)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("opt", ["", "cap", "slopes", "sinks", "other", "cap slopes sinks other"])
def test_attn_options(opt, dtype):
    rng = np.random.default_rng(len(opt))
    rows = [400, 0, 130, 129, 1, 77]
    pool = Pool(rng, rows, 16, dtype)
    q = queries(rng, 6, dtype)
    opts = options(rng, 6, dtype, **{k: True for k in opt.split()})
    out, lse = run_attn(q, pool, opts, {})
    check_attn(q, pool, out, lse, dtype, SCALE, opts, {})


@pytest.mark.parametrize("cap", [1e-42, 1e-30, 0.3, 20.0, 255.0, 257.0, 5e3, 1e7, 1e30, 3.4e38])
def test_attn_cap(cap):
    """Caps from none of the logits to all of them: a large one leaves them as they are, to fp32's last places."""
    rng = np.random.default_rng(6)
    pool = Pool(rng, [500, 90], 16, "f16", size=3.0)
    q = queries(rng, 2, "f16", size=8.0)
    opts = dict(cap=float(np.float32(cap)))
    out, lse = run_attn(q, pool, opts, {})
    check_attn(q, pool, out, lse, "f16", SCALE, opts, {})


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("window", [1, 7, 64, 127, 128, 129, 200, 1000])
def test_attn_window(window, dtype):
    """Chunks of three requests whose pages before the chunk's first window are gone, sinks and a join."""
    rng = np.random.default_rng(window)
    rows, per, ps = [300, 40, 517], 23, 16
    pos = np.concatenate([np.arange(n - per, n) for n in rows])
    gone = [max(0, n - per + 1 - window) for n in rows]
    pool = Pool(rng, rows, ps, dtype, gone=gone)
    lists = dict(req=np.repeat(np.arange(3), per), positions=pos, window=window)
    q = queries(rng, 3 * per, dtype)
    opts = options(rng, 3 * per, dtype, sinks=True, other=True)
    out, lse = run_attn(q, pool, opts, lists)
    check_attn(q, pool, out, lse, dtype, SCALE, opts, lists, tokens=range(0, 3 * per, 4))
    check_attn(q, pool, out, lse, dtype, SCALE, opts, lists, tokens=range(3 * per - 3, 3 * per))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attn_masks_that_meet(dtype):
    """Documents, a prefix, a window, negative positions, requests that are none, rows not held yet."""
    rng = np.random.default_rng(8)
    rows = [260, 33, 0, 150]
    pool = Pool(rng, rows, 8, dtype)
    T = 40
    req = rng.integers(-1, 6, T)
    pos = rng.integers(-2, 300, T)
    first = np.where(rng.random(T) < 0.5, 0, rng.integers(0, 280, T))
    first[3] = -5
    lists = dict(req=req, positions=pos, first=first, prefix=np.array([90, 50, 7, -3]), window=120)
    q = queries(rng, T, dtype)
    opts = options(rng, T, dtype, slopes=True, cap=True)
    out, lse = run_attn(q, pool, opts, lists)
    check_attn(q, pool, out, lse, dtype, SCALE, opts, lists)
    assert torch.isneginf(lse).all(1).any()                       # some token saw nothing
    for drop in ("first", "prefix", "window"):
        some = {k: v for k, v in lists.items() if k != drop}
        out, lse = run_attn(q, pool, opts, some)
        check_attn(q, pool, out, lse, dtype, SCALE, opts, some, tokens=range(0, T, 3))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("ps", [4, 8, 16, 32, 64, 512])
def test_attn_long_lists(ps, dtype):
    """Lists long enough to be cut at multiples of 64 rows, that begin and end anywhere, in pages of any size; rows
    whose pages are gone; the same lists a row too short for it."""
    rng = np.random.default_rng(ps)
    rows = [1500, 700, 1024]
    pool = Pool(rng, rows, ps, dtype, gone=[0, 130, 0])
    pool.tables[2, 300 // ps] = -1
    pool.dev = pool.dev[0], i32(pool.tables), pool.dev[2]
    req = np.array([0, 0, 0, 0, 0, 1, 1, 1, 2, 2, 2])
    pos = np.array([1499, 1023, 1024, 511, 510, 699, 650, 1400, 1023, 1022, 1000])
    first = np.array([0, 1, 513, 0, 0, 60, 139, 0, 0, 511, 128])
    q = queries(rng, len(req), dtype)
    for opts in ({}, options(rng, len(req), dtype, slopes=True, cap=True, other=True)):
        lists = dict(req=req, positions=pos, first=first)
        out, lse = run_attn(q, pool, opts, lists)
        check_attn(q, pool, out, lse, dtype, SCALE, opts, lists)
    lists = dict(req=req, positions=pos, first=first, prefix=np.array([600, 0, 0]), window=620)
    out, lse = run_attn(q, pool, {}, lists)
    check_attn(q, pool, out, lse, dtype, SCALE, {}, lists)


@pytest.mark.parametrize("ratio", [4, 128])
def test_attn_pooled_rows(ratio):
    """Rows of several positions each: the ratio of the pooled rows."""
    rng = np.random.default_rng(ratio)
    rows = [70, 300]
    pool = Pool(rng, rows, 32, "bf16")
    pos = np.array([0, ratio - 1, 70 * ratio - 1, 69 * ratio, 5, 299 * ratio, 300 * ratio - 1, 2 ** 31 - 1])
    lists = dict(req=[0, 0, 0, 0, 1, 1, 1, 1], positions=pos, ratio=ratio, window=150)
    q = queries(rng, 8, "bf16")
    opts = options(rng, 8, "bf16", slopes=True)
    out, lse = run_attn(q, pool, opts, lists)
    check_attn(q, pool, out, lse, "bf16", SCALE, opts, lists)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attn_loud_logits(dtype):
    """Logits of some hundreds, whose maximum moves from chunk to chunk, and biases that dwarf them."""
    rng = np.random.default_rng(4)
    pool = Pool(rng, [900, 700], 64, dtype, size=6.0)
    q = queries(rng, 2, dtype, size=20.0)
    for opts in ({}, dict(slopes=np.float32(np.linspace(0, 40, 64)))):
        out, lse = run_attn(q, pool, opts, {})
        check_attn(q, pool, out, lse, dtype, SCALE, opts, {})
    up = dict(slopes=np.float32(np.linspace(0, -40, 64)))          # far rows count most
    out, lse = run_attn(q, pool, up, {})
    check_attn(q, pool, out, lse, dtype, SCALE, up, {})


@pytest.mark.parametrize("T,rows", [(1, 20001), (3, 3000), (40, 900), (37, 2600), (160, 300)])
def test_attn_splits(T, rows):
    """Few tokens over many rows, many over some: tokens whose rows lie in several blocks."""
    rng = np.random.default_rng(T)
    n = rng.integers(1, rows + 1, T)
    n[0] = rows
    pool = Pool(rng, n, 64, "bf16")
    q = queries(rng, T, "bf16")
    opts = options(rng, T, "bf16", sinks=True, other=True)
    out, lse = run_attn(q, pool, opts, {})
    check_attn(q, pool, out, lse, "bf16", SCALE, opts, {}, tokens=range(0, T, max(1, T // 12)))
    again, _ = run_attn(q, pool, opts, {})
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("rows", [
    [3000] * 4,                       # two dozen parts a token
    [1, 20000, 300, 5, 9000] + [64] * 4,
    [5 * 3 ** (i % 9) for i in range(40)],
    [1000] * 9 + [20000] + [300] * 120,   # fewer tokens than blocks, one of them over most of these
    [70] * 100 + [9000] + [260] * 120,    # more tokens than blocks, one of them over several
    [33000, 5],
], ids=["even", "two-long", "ragged", "one-over-many", "one-among-many", "long-and-short"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attn_parts(rows, dtype):
    """However many parts a token has, and however many tokens have some: out and lse are whole, and the same again."""
    rng = np.random.default_rng(len(rows))
    T = len(rows)
    pool = Pool(rng, rows, 64, dtype)
    q = queries(rng, T, dtype)
    opts = options(rng, T, dtype, sinks=True, cap=True)
    out, lse = run_attn(q, pool, opts, {})
    longest = int(np.argmax(rows))
    check_attn(q, pool, out, lse, dtype, SCALE, opts, {}, tokens={0, longest, max(longest - 1, 0), *range(1, T, max(1, T // 6)), T - 1})
    again, lse2 = run_attn(q, pool, opts, {})
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attn_lists_of_several_items(dtype):
    """A block with tens of thousands of a token's rows, whole or in part, adds them up in several goes."""
    rng = np.random.default_rng(17)
    T, rows = 160, 35000
    pool = Pool(rng, [rows], 512, dtype)
    lists = dict(req=np.zeros(T, np.int32), positions=np.arange(rows - T, rows))
    q = queries(rng, T, dtype)
    opts = options(rng, T, dtype, sinks=True, slopes=True, other=True)
    out, lse = run_attn(q, pool, opts, lists)
    check_attn(q, pool, out, lse, dtype, SCALE, opts, lists, tokens=[0, 80])


def test_attn_chunk_of_many_tokens():
    """More tokens than one launch plans for, over a causal chunk."""
    rng = np.random.default_rng(6)
    T = 2300
    pool = Pool(rng, [T], 32, "bf16")
    lists = dict(req=np.zeros(T, np.int32), positions=np.arange(T), window=200, first=np.arange(T) // 701 * 701)
    q = queries(rng, T, "bf16")
    out, lse = run_attn(q, pool, {}, lists)
    check_attn(q, pool, out, lse, "bf16", SCALE, {}, lists,
               tokens=[0, 1, 127, 128, 200, 700, 701, 702, 1500, 2047, 2048, 2049, 2299])


def test_attn_nan_rows():
    """A NaN row reaches the tokens that see it and no others."""
    rng = np.random.default_rng(5)
    pool = Pool(rng, [200, 200], 16, "bf16")
    bad = pool.tables[0, 150 // 16] * 16 + 150 % 16
    pool.dev[0][bad, 100] = float("nan")
    pos = np.array([149, 150, 151, 199, 199])
    lists = dict(req=[0, 0, 0, 0, 1], positions=pos, window=49)
    q = queries(rng, 5, "bf16")
    out, lse = run_attn(q, pool, {}, lists)
    assert torch.isnan(lse).all(1).tolist() == [False, True, True, False, False]     # 199 - 49 + 1 = 151
    assert torch.isfinite(out).all(2).all(1).tolist() == [True, False, False, True, True]
    check_attn(q, pool, out, lse, "bf16", SCALE, {}, lists, tokens=[0, 3, 4])


def test_attn_nothing_to_see():
    q = torch.randn((3, 64, 512), device="cuda").half()
    pool = torch.full((64, 512), float("nan"), dtype=torch.float16, device="cuda")
    z = i32([0, 0, 0])
    for tables, rows in ((i32([[0], [1], [2]]), z), (i32([[-1], [-1], [-1]]), i32([9, 9, 9])),
                         (i32([[77], [64], [100]]), i32([9, 9, 9])), (torch.empty((3, 0), dtype=I32, device="cuda"), z)):
        out, lse = ds4x.kv16_attn(q, pool, tables, rows, 16)
        assert (out == 0).all() and torch.isneginf(lse).all()
    sinks = torch.randn(64, device="cuda")
    out, lse = ds4x.kv16_attn(q, pool, i32([[0], [1], [2]]), z, 16, sinks=sinks)
    assert (out == 0).all() and (lse - sinks).abs().max() <= 2.0 ** -20
    o, l = torch.randn((3, 64, 512), device="cuda").half(), torch.randn((3, 64), device="cuda")
    out, lse = ds4x.kv16_attn(q, pool, i32([[0], [1], [2]]), z, 16, other=(o, l))
    assert (out.float() - o.float()).abs().max() <= 2.0 ** -9 and (lse - l).abs().max() <= 2.0 ** -20
    out, lse = ds4x.kv16_attn(q[:0], pool, i32([[0]]), i32([4]), 16)
    assert out.shape == (0, 64, 512) and lse.shape == (0, 64)
    out, lse = ds4x.kv16_attn(q[:1], pool[:0], i32([[0]]), i32([4]), 16)
    assert (out == 0).all()


@pytest.mark.parametrize("low", [-1e3, -1e30, float(np.finfo(np.float32).min)])
def test_attn_other_of_next_to_no_weight(low):
    """A finite lse as low as the type has counts alone, and for nothing beside rows."""
    q, pool = torch.randn((2, 64, 512), device="cuda").bfloat16(), torch.randn((32, 512), device="cuda").bfloat16()
    other = torch.randn((2, 64, 512), device="cuda").bfloat16(), torch.full((2, 64), low, device="cuda")
    out, lse = ds4x.kv16_attn(q, pool, i32([[0], [1]]), i32([0, 7]), 16, other=other)
    want, wlse = ds4x.kv16_attn(q, pool, i32([[0], [1]]), i32([0, 7]), 16)
    assert (out[0].float() - other[0][0].float()).abs().max() <= 2.0 ** -7
    assert lse[0].max() < 0.6 * low
    # weights against another offset, each rounded on its own: two half steps of numbers of order one each
    assert (out[1].float() - want[1].float()).abs().max() <= 4 * 2.0 ** -8 * pool.float().abs().max()
    assert (lse[1] - wlse[1]).abs().max() <= 2.0 ** -18


def test_attn_writes_its_tokens_only():
    rng = np.random.default_rng(2)
    pool = Pool(rng, [300, 200], 16, "f16")
    q = queries(rng, 2, "f16")
    buf = torch.full((4, 64, 512), 7.0, dtype=torch.float16, device="cuda")
    lb = torch.full((4, 64), 7.0, device="cuda")
    run_attn(q, pool, {}, {}, out=buf[1:3], lse=lb[1:3])
    want, wl = run_attn(q, pool, {}, {})
    assert torch.equal(buf[1:3], want) and torch.equal(lb[1:3], wl)
    assert (buf[[0, 3]] == 7).all() and (lb[[0, 3]] == 7).all()
    alone, none = run_attn(q, pool, {}, {}, want_lse=False)
    assert none is None and torch.equal(alone, want)


def test_rows_far_into_a_large_pool():
    """Slots whose elements lie beyond 2^31, and beyond 2^32 bytes."""
    n_slots = (1 << 22) + 4096
    pool = torch.empty((n_slots, 512), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((130, 512))).bfloat16().cuda()
    slots = torch.arange(n_slots - 130, n_slots, dtype=I32, device="cuda")
    ds4x.kv16_append(x, slots, pool)
    assert torch.equal(pool[-130:], x)
    small = torch.zeros((192, 512), dtype=torch.bfloat16, device="cuda")
    small[62:] = x
    q = queries(rng, 1, "bf16")
    first = i32([62])
    a = ds4x.kv16_attn(q, pool, i32([[n_slots // 64 - 3, n_slots // 64 - 2, n_slots // 64 - 1]]), i32([192]), 64, first=first)
    b = ds4x.kv16_attn(q, small, i32([[0, 1, 2]]), i32([192]), 64, first=first)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_many_tokens_beyond_32_bit_offsets():
    T = 66000                                                      # 2.16e9 elements
    pool = torch.randn((64, 512), device="cuda").half()
    q = torch.zeros((T, 64, 512), dtype=torch.float16, device="cuda")
    q[-1] = torch.randn((64, 512), device="cuda").half()
    req = torch.zeros(T, dtype=I32, device="cuda")
    pos = torch.arange(T, device="cuda", dtype=I32) % 64
    out, lse = ds4x.kv16_attn(q, pool, i32([[0]]), i32([64]), 64, req=req, positions=pos, window=2)
    one, l1 = ds4x.kv16_attn(q[-1:].clone(), pool, i32([[0]]), i32([64]), 64, req=req[:1], positions=pos[-1:], window=2)
    assert torch.equal(out[-1], one[0]) and torch.equal(lse[-1], l1[0])
    mean = (pool[61].float() + pool[62].float()) / 2               # a query of zeros: the mean of its two rows
    t = 62 + 64 * 1030
    assert (out[t].float() - mean).abs().max() <= 2.0 ** -10 * 1.01 * mean.abs().max()
    back = ds4x.rotate(out, pos, gpu(frequencies(64)), out=out)
    assert torch.isfinite(back[-1]).all()


# ------------------------------------------------------------------------ as they are used together
def test_captured_step_and_two_streams():
    """A captured step replayed on new values, and two calls at once on streams of their own."""
    rng = np.random.default_rng(12)
    pool = Pool(rng, [500] * 5, 16, "bf16")
    f = gpu(frequencies(64))
    q, x = queries(rng, 5, "bf16"), torch.randn((5, 512), device="cuda").bfloat16()
    slots = i32([pool.tables[b, 499 // 16] * 16 + 499 % 16 for b in range(5)])
    pos = i32([499] * 5)
    req = i32(range(5))

    def step():
        ds4x.kv16_append(x, slots, pool.dev[0], positions=pos, inv_freq=f)
        out, lse = ds4x.kv16_attn(ds4x.rotate(q, pos, f), *pool.dev, 16, req=req, positions=pos)
        return ds4x.rotate(out, pos, f, inverse=True), lse
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(3):
        q.copy_(torch.randn_like(q))
        x.copy_(torch.randn_like(x))
        g.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in got]
        want = step()
        assert torch.equal(replayed[0], want[0]) and torch.equal(replayed[1], want[1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    qs = [queries(rng, 5, "bf16") for _ in range(2)]
    want = [ds4x.kv16_attn(a, *pool.dev, 16) for a in qs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [ds4x.kv16_attn(a, *pool.dev, 16, stream=s) for a, s in zip(qs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def capture_after_another_call():
    """A short call, then captures of calls that take other kernels: more types, caps, and every way of joining."""
    rng = np.random.default_rng(14)
    for dtype in ("bf16", "f16"):
        small = Pool(rng, [5], 16, "bf16")
        ds4x.kv16_attn(queries(rng, 1, "bf16"), *small.dev, 16)
        for T, rows, cap in ((1, 3000, 0.0), (9, 1200, 0.7), (200, 300, 900.0)):
            pool = Pool(rng, [rows] * T, 64, dtype)
            q = queries(rng, T, dtype)
            x, f, pos = torch.zeros((T, 512), dtype=q.dtype, device="cuda"), gpu(frequencies(64)), i32([7] * T)
            slots = i32([-1] * T)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                ds4x.kv16_append(x, slots, pool.dev[0], positions=pos, inv_freq=f)
                got = ds4x.kv16_attn(ds4x.rotate(q, pos, f), *pool.dev, 64, cap=cap)
            g.replay()
            torch.cuda.synchronize()
            want = ds4x.kv16_attn(ds4x.rotate(q, pos, f), *pool.dev, 64, cap=cap)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (dtype, T)
    assert ds4x.device_status() == ds4x.OK


def test_capture_after_another_call():
    """In a process of its own, whose kernels no other test has brought to the device."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = "from tests.test_gpu_kv16 import capture_after_another_call as f; f()"
    got = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0, got.stderr[-2000:]


def test_graphs_that_share_a_workspace():
    """Nothing is kept in it: two captured graphs use one in turn."""
    rng = np.random.default_rng(15)
    pools = [Pool(rng, [2500] * 3, 64, "bf16"), Pool(rng, [700] * 30, 64, "bf16")]
    qs = [queries(rng, 3, "bf16"), queries(rng, 30, "bf16")]
    work = torch.full((max(ds4x.kv16_attn_workspace_bytes(len(q), p.max_pages * 64) for q, p in zip(qs, pools)),), 0xff,
                      dtype=torch.uint8, device="cuda")
    want = [ds4x.kv16_attn(q, *p.dev, 64) for q, p in zip(qs, pools)]
    torch.cuda.synchronize()
    graphs, got = [], []
    for q, p in zip(qs, pools):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(ds4x.kv16_attn(q, *p.dev, 64, workspace=work))
        graphs.append(g)
    for i in (0, 1, 1, 0, 1):
        got[i][0].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1])


def test_a_serving_step_of_both_caches():
    """Two steps of a batch: plans of both caches, raw rows rotated into the 16-bit one, pooled rows into the 4-bit
    one, attention over both in one softmax, and the outputs turned back."""
    rng = np.random.default_rng(21)
    B, ratio, ps, rps, window = 4, 4, 8, 16, 50
    f = frequencies(64)
    df = gpu(f)
    dt = torch.bfloat16
    mk = lambda n, p: (torch.full((B, n), -1, dtype=I32, device="cuda"),  # noqa: E731
                       i32(rng.permutation(p)), i32([p]))
    tab, free, n_free = mk(12, 60)
    rtab, rfree, rn_free = mk(24, 100)
    codes = torch.zeros((60 * ps, 256), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((60 * ps, 16), dtype=torch.uint8, device="cuda")
    raw = torch.full((100 * rps, 512), float("nan"), dtype=dt, device="cuda")
    seen = i32([0] * B)
    rows, rrows = i32([0] * B), i32([0] * B)
    history = [np.zeros((0, 512)) for _ in range(B)]
    pooled = [np.zeros((0, 512)) for _ in range(B)]
    for new in ([70, 1, 0, 33], [1, 60, 5, 200]):
        T = sum(new) + 3
        R = T // ratio + B
        x = torch.from_numpy(rng.standard_normal((T, 512))).to(dt).cuda()
        p4 = torch.from_numpy(rng.standard_normal((R, 512))).to(dt).cuda()
        q = queries(rng, T, "bf16")
        nn = i32(new)
        rp = ds4x.page_plan(seen, nn, rrows, rtab, rfree, rn_free, 1, rps, T, T)
        pos, req, rslots = rp[:3]
        pp = ds4x.page_plan(seen, nn, rows, tab, free, n_free, ratio, ps, T, R)
        ds4x.kv16_append(x, rslots, raw, positions=pos, inv_freq=df)
        ds4x.kv4_append(p4, pp[2], codes, scales)
        seen, rrows, rn_free = rp[3], rp[4], rp[5]
        rows, n_free = pp[4], pp[5]
        qr = ds4x.rotate(q, pos, df)
        part = ds4x.kv4_attn(qr, codes, scales, tab, rows, ps, req=req, positions=pos, ratio=ratio)
        out, lse = ds4x.kv16_attn(qr, raw, rtab, rrows, rps, req=req, positions=pos, window=window, other=part)
        back = ds4x.rotate(out, pos, df, inverse=True)
        # the same from the definitions, in 64 bits on the operands as the caches hold them
        hp, hr, hs = (t.cpu().numpy() for t in (pos, req, pp[2]))
        stored = raw.double().cpu().numpy()[np.maximum(rslots.cpu().numpy(), 0)]
        vals = kv4.values(codes.cpu().numpy(), scales.cpu().numpy())
        for t in range(T):
            if hr[t] >= 0:
                history[hr[t]] = np.concatenate([history[hr[t]], stored[t:t + 1]])
        ends = np.cumsum([(s + n) // ratio - s // ratio for s, n in zip(before_of(hp, hr, B, new, seen), new)])
        k = 0
        for b in range(B):
            while k < ends[b]:
                pooled[b] = np.concatenate([pooled[b], vals[hs[k]][None]])
                k += 1
        qd = qr.double().cpu().numpy()
        go, gl, gb = (t.double().cpu().numpy() for t in (out, lse, back))
        assert np.all(hr[-3:] == -1) and np.all(go[-3:] == 0) and np.all(np.isneginf(gl[-3:]))
        for t in range(T - 3):
            b, p = hr[t], hp[t]
            kv = np.concatenate([pooled[b][:(p + 1) // ratio], history[b][max(0, p + 1 - window):p + 1]])
            lg = qd[t] @ kv.T * SCALE
            m = lg.max(1, keepdims=True)
            w = np.exp(lg - m)
            ref = w @ kv / w.sum(1, keepdims=True)
            # weights and the pooled part's output are rounded to bf16 on the way, the output once more
            spread = np.stack([(w[h] / w[h].sum()) @ np.abs(kv - ref[h]) for h in range(64)])
            tol = 2.0 ** -8 * (2.2 * spread + 2.1 * np.abs(ref) + 0.01 * np.abs(kv).max())
            assert np.all(np.abs(go[t] - ref) <= tol + 2.0 ** -8 * 0.2), t
            assert np.all(np.abs(gl[t] - (m[:, 0] + np.log(w.sum(1)))) <= 1e-4)
            turned = kv16.rotate(go[t][None], [p], f, inverse=True)[0]
            assert np.all(np.abs(gb[t] - turned) <= 2.0 ** -8 * 1.01 * np.abs(turned) + 2.0 ** -20 * 4)


def before_of(positions, req, B, new, seen):
    """Positions of each request before the step."""
    return [int(s) - n for s, n in zip(seen.cpu().numpy(), new)]


def test_agrees_with_the_dense_window_attention():
    """One request: the pooled rows from the 4-bit cache, the window from the 16-bit one, against the dense entry."""
    rng = np.random.default_rng(33)
    S, T, window, L = 96, 12, 40, 400
    codes = gpu(rng.integers(0, 256, (S, 256), dtype=np.uint8))
    scales = gpu(rng.integers(124, 127, (S, 16), dtype=np.uint8))
    kv = ds4x.kv4_read(codes, scales, i32(range(S)), torch.bfloat16)
    raw = torch.randn((L, 512), device="cuda").bfloat16()
    pos = np.arange(L - T, L)
    q = queries(rng, T, "bf16")
    idx = np.sort(np.stack([rng.permutation(S)[:64] for _ in range(T)]), axis=1)
    req = i32([0] * T)
    dense, dlse = ds4x.local_pooled_attn(q, kv, raw, i32(idx), i32(pos), 0, window)
    part = ds4x.kv4_attn(q, codes, scales, i32([[0]]), i32([S]), 128, req=req, indices=i32(idx))
    out, lse = ds4x.kv16_attn(q, raw, i32([range(L // 16)]), i32([L]), 16, req=req, positions=i32(pos), window=window,
                              other=part)
    # each side rounds weights, parts and outputs to bf16: a few half steps of numbers of order one
    assert (out.float() - dense.float()).abs().max() <= 4 * 2.0 ** -8
    assert (lse - dlse).abs().max() <= 4 * 2.0 ** -8


def test_refusals_on_the_device():
    q = torch.zeros((2, 64, 512), dtype=torch.float16, device="cuda")
    pool = torch.zeros((32, 512), dtype=torch.float16, device="cuda")
    tab, rows = i32([[0], [1]]), i32([3, 3])
    call = lambda **kw: ds4x.kv16_attn(q, pool, tab, rows, 16, **kw)  # noqa: E731
    for bad in (dict(positions=i32([1])), dict(first=i32([0])), dict(prefix=i32([0])), dict(req=torch.zeros(2, device="cuda")),
                dict(sinks=torch.zeros(3, device="cuda")), dict(slopes=torch.zeros(64, dtype=torch.float64, device="cuda")),
                dict(other=(q[:1], torch.zeros((2, 64), device="cuda"))), dict(out=q[:1]), dict(window=-1), dict(ratio=0),
                dict(window=1 << 40), dict(other=(q.bfloat16(), torch.zeros((2, 64), device="cuda")))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(ds4x.Ds4xError):
        call(cap=-1.0)
    with pytest.raises(ValueError):
        ds4x.kv16_attn(q, pool.bfloat16(), tab, rows, 16)
    with pytest.raises(ValueError):
        ds4x.kv16_attn(q.transpose(1, 2).contiguous().transpose(1, 2), pool, tab, rows, 16)
    assert ds4x.kv16_attn_workspace_bytes(2, 16) == 0
    long = i32([[0] * 64] * 2)  # 1024 rows may be split over blocks
    assert ds4x.kv16_attn_workspace_bytes(2, 1024) > 8
    with pytest.raises(ds4x.Ds4xError):
        ds4x.kv16_attn(q, pool, long, rows, 16, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    f = torch.zeros(32, dtype=torch.float64, device="cuda")
    with pytest.raises(ValueError):
        ds4x.rotate(q, rows, f.float())
    with pytest.raises(ValueError):
        ds4x.rotate(q, rows[:1], f)
    with pytest.raises(ValueError):
        ds4x.kv16_append(q[0], rows, pool)                        # 64 rows, two slots
    with pytest.raises(ValueError):
        ds4x.kv16_append(q[0, :2], rows, pool, inv_freq=f)
    with pytest.raises(ds4x.Ds4xError):
        ds4x.rotate(q, rows, f[:0])


# --------------------------------------------------------------------- the ends of the ranges
LOWEST = float(np.finfo(np.float32).min)
LOW = [LOWEST, -3e38, -2.4e38, -1e38, -1e30, -np.inf]
HIGH = [1e30, 1e38, 2.3e38, 2.4e38, 3e38, -LOWEST]
# whole tokens and split ones, joined each of the three ways; the second sees no row
ENDS = [[40, 0], [3000, 0, 40], [20000, 0] + [300] * 7, [260] * 160]


def heads_of(values):
    return np.float32([values[h % len(values)] for h in range(64)])


def ends_pool(rng, rows, dtype):
    rows = [rows[0], 0, *rows[2:]]
    return Pool(rng, rows, 64, dtype), queries(rng, len(rows), dtype)


def nearly(a, b):
    """Equal but for a few fp32 steps, infinities too."""
    b = torch.as_tensor(b, device=a.device).expand_as(a)
    return bool(((a == b) | ((a.double() - b.double()).abs() <= 2.0 ** -21 * b.double().abs())).all())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows", ENDS, ids=["whole", "few", "some", "many"])
def test_attn_sinks_at_the_ends_of_fp32(rows, dtype):
    """A sink of next to no weight is none beside rows and all there is without; one above all logits is all there is."""
    rng = np.random.default_rng(31)
    pool, q = ends_pool(rng, rows, dtype)
    without, wlse = run_attn(q, pool, dict(sinks=heads_of([-np.inf])), {})
    assert torch.isfinite(wlse[0]).all() and torch.isneginf(wlse[1]).all()
    out, lse = run_attn(q, pool, dict(sinks=heads_of(LOW)), {})
    assert torch.equal(out, without)
    assert torch.equal(lse[0], wlse[0]) and torch.equal(lse[2:], wlse[2:]) and nearly(lse[1], gpu(heads_of(LOW)))
    out, lse = run_attn(q, pool, dict(sinks=heads_of(HIGH)), {})
    assert (out == 0).all() and nearly(lse, gpu(heads_of(HIGH)))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows", ENDS, ids=["whole", "few", "some", "many"])
def test_attn_other_at_the_ends_of_fp32(rows, dtype):
    """The same of another attention's log-sum-exp, whose output counts with it."""
    rng = np.random.default_rng(32)
    pool, q = ends_pool(rng, rows, dtype)
    T = len(q)
    oo = torch.from_numpy(rng.standard_normal((T, 64, 512))).to(DT[dtype]).cuda()
    with_lse = lambda v: run_attn(q, pool, dict(other=(oo, gpu(heads_of(v)).expand(T, 64).contiguous())), {})  # noqa: E731
    without, wlse = with_lse([-np.inf])
    assert torch.isfinite(wlse[0]).all() and torch.isneginf(wlse[1]).all() and (without[1] == 0).all()
    out, lse = with_lse(LOW)
    alone = gpu(np.isfinite(heads_of(LOW)))[:, None]
    seen = [t for t in range(T) if t != 1]
    assert torch.equal(out[seen], without[seen]) and torch.equal(lse[seen], wlse[seen])
    assert torch.equal(out[1], torch.where(alone, oo[1], 0)) and nearly(lse[1], gpu(heads_of(LOW)))
    out, lse = with_lse(HIGH)
    assert torch.equal(out, oo) and nearly(lse, gpu(heads_of(HIGH)))


@pytest.mark.parametrize("rows", ENDS, ids=["whole", "few", "some", "many"])
def test_attn_sinks_and_other_at_the_ends_of_fp32(rows):
    """The larger of a sink and another attention takes all; equal ones take half each."""
    rng = np.random.default_rng(33)
    pool, q = ends_pool(rng, rows, "bf16")
    T = len(q)
    oo = torch.from_numpy(rng.standard_normal((T, 64, 512))).bfloat16().cuda()
    for values, seen in ((HIGH, range(T)), (LOW[:5], [1])):
        pairs = [(a, b) for a in values for b in values]
        s, o = heads_of([a for a, _ in pairs]), heads_of([b for _, b in pairs])
        out, lse = run_attn(q, pool, dict(sinks=s, other=(oo, gpu(o).expand(T, 64).contiguous())), {})
        share = gpu(np.float32(np.where(s < o, 1, np.where(s == o, 0.5, 0))))[:, None]
        for t in seen:
            assert torch.equal(out[t].float(), oo[t].float() * share) and nearly(lse[t], gpu(np.maximum(s, o)))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [[40], [3000, 700], [20000] + [300] * 8, [260] * 160], ids=["whole", "few", "some", "many"])
def test_attn_slopes_at_the_end_of_fp32(rows, dtype):
    """A slope that leaves nothing but the row at distance 0, capped logits and others."""
    rng = np.random.default_rng(34)
    pool, q = Pool(rng, rows, 64, dtype), queries(rng, len(rows), dtype)
    near = dict(first=np.asarray(rows) - 1)
    for cap in (0.0, 1.5, 900.0):
        out, lse = run_attn(q, pool, dict(slopes=heads_of([2.3e38, 2.4e38, 3e38, -LOWEST]), cap=cap), {})
        one, olse = run_attn(q, pool, dict(cap=cap), near)
        assert torch.equal(out, one) and torch.equal(lse, olse)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("cap", [0.0, 1.5, 400.0])
@pytest.mark.parametrize("scale", [0.0, 0.003, 0.09, 0.7, -0.05])
def test_attn_scale(scale, cap, dtype):
    """Scales of the caller's own: with a cap they take another way through the kernel."""
    rng = np.random.default_rng(35)
    rows = [400, 0, 130, 1, 77, 1500]
    pool = Pool(rng, rows, 16, dtype)
    q = queries(rng, len(rows), dtype)
    opts = options(rng, len(rows), dtype, slopes=True, sinks=True)
    for o in ({}, opts):
        o = dict(o, cap=cap) if cap else o
        out, lse = run_attn(q, pool, o, {}, scale=scale)
        check_attn(q if scale >= 0 else -q, pool, out, lse, dtype, abs(scale), o, {})


# ------------------------------------------------------- every part and item of a long list counts
class MarkedPool(Pool):
    """One request, whose rows are quiet but for one value: 64 at element r // group % 512 of row r.  With weights that
    are about equal, the rows of a group are all there is of their element of the output."""
    MARK = 64.0

    def __init__(self, rng, rows, group, dtype, ps=64):
        n_pages = -(-rows // ps)
        self.ps, self.n_slots, self.rows, self.group = ps, n_pages * ps, np.array([rows], dtype=np.int32), group
        self.tables = rng.permutation(n_pages).astype(np.int32)[None, :]
        self.kv = (torch.randn((rows, 512), generator=torch.Generator("cuda").manual_seed(rows), device="cuda") * 0.1)
        r = torch.arange(rows, device="cuda")
        self.kv[r, r // group % 512] = self.MARK
        self.kv = self.kv.to(DT[dtype])
        pool = torch.full((self.n_slots, 512), float("nan"), dtype=DT[dtype], device="cuda")
        pool[i32(self.tables)[0].long()[r // ps] * ps + r % ps] = self.kv
        self.dev = pool, i32(self.tables), i32(self.rows)


def check_marked(pool, q, out, lse, dtype, lo, hi, opts, tokens):
    """Token t over rows [lo[t], hi[t]), which end at e = hi[t], against plain sums in 64 bits.  Every whole group of rows
    has to be worth four tolerances at its element at least, so that none can be lost, or be off by a quarter."""
    u = torch.finfo(DT[dtype]).eps / 2
    for t in tokens:
        kv = pool.kv[lo[t]:hi[t]].double()
        n = len(kv)
        x = q[t].double() @ kv.T * SCALE
        # 512 exact products summed in fp32 by a truncating adder, and 2^x with its argument
        ex = 64 * 2.0 ** -23 * SCALE * (q[t].double().abs() @ kv.abs().T).max() + 2.0 ** -20 + 2.0 ** -22 * x.abs().max()
        if "slopes" in opts:
            away = torch.arange(n - 1, -1, -1, device="cuda").double()
            x -= gpu(opts["slopes"]).double()[:, None] * away
            ex += 2.0 ** -22 * x.abs().max()
        extra = [gpu(opts["sinks"]).double()] if "sinks" in opts else []
        if "other" in opts:
            oo, ol = (v[t].double() for v in opts["other"])
            extra.append(ol)
        want = torch.logsumexp(torch.cat([x] + [v[:, None] for v in extra], 1), 1)
        w = torch.exp(x - want[:, None])
        ref, size = w @ kv, w @ kv.abs()
        if "other" in opts:
            share = torch.exp(ol - want)[:, None]
            ref, size = ref + share * oo, size + share * oo.abs()
        # A weight is rounded to half a step u, and off by ex twice, in numerator and normaliser; |kv - ref| <= |kv| + |ref|.
        # The matrix unit truncates fp32 sums, one a step of 16 rows and 1024 in a row at most, as many as 256 parts and the
        # threads' own sums are added to with roundings.  Weights are 2^4 times 2^(x - an offset that no maximum is below),
        # in fp16 those below its normal range off by 2^-25, which is 2^-29 of the largest.
        tol = 2 * (u + 2 * ex) * (size + ref.abs()) + (1024 + 256) * 2.0 ** -23 * size + u * 1.01 * ref.abs() + 2.0 ** -25
        if dtype == "f16":
            total = torch.exp(want - torch.maximum(x.amax(1), torch.stack(extra).amax(0)) if extra else want - x.amax(1))
            tol += 2.0 ** -29 / total[:, None] * (kv.abs().sum(0) + n * ref.abs())
        g0, g1 = -(-lo[t] // pool.group), hi[t] // pool.group
        if g1 > g0:
            part = w[:, g0 * pool.group - lo[t]:g1 * pool.group - lo[t]].reshape(64, g1 - g0, pool.group).sum(2) * pool.MARK
            at = torch.arange(g0, g1, device="cuda") % 512
            assert (part > 4 * tol[:, at]).all(), (t, (part / tol[:, at]).min().item())
        worst = ((out[t].double() - ref).abs() / tol).max().item()
        assert worst <= 1, (t, n, worst)
        assert ((lse[t].double() - want).abs() <= 2 * ex + 2.0 ** -15).all(), t


def flat_queries(rng, T, dtype):
    """Logits of a tenth: the rows' marks of 64 times these and 512^-1/2."""
    return queries(rng, T, dtype, size=0.03)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens", [
    [33000], [2900, 33000, 5], [3000] * 4, [700] * 12, [20000, 300, 5, 9000] + [64] * 5, [5 * 3 ** (i % 9) for i in range(37)],
    [1000] * 9 + [20000] + [300] * 120, [70] * 100 + [9000] + [260] * 120, [901] * 200,
], ids=["few-one", "few-three", "some-even", "some-short", "some-two-long", "some-ragged", "some-one-over-many", "many-one-long",
        "many-even"])
def test_attn_every_part_counts(lens, dtype):
    """Each chunk of 64 rows shows in the output, whichever block and way of joining it goes through."""
    rng = np.random.default_rng(sum(lens))
    T, rows = len(lens), max(lens) + 100
    pool = MarkedPool(rng, rows, 64, dtype)
    hi = np.array([rng.integers(n, rows + 1) for n in lens])
    lo = hi - lens
    lists = dict(req=np.zeros(T, np.int32), positions=hi - 1, first=lo)
    q = flat_queries(rng, T, dtype)
    n = np.log(np.asarray(lens))
    other = (torch.randn((T, 64, 512), device="cuda") * 0.1).to(DT[dtype]), gpu(np.float32(n[:, None] - rng.uniform(0, 3, (T, 64))))
    for opts in ({}, dict(sinks=np.float32(rng.uniform(0, n.min(), 64)), other=other)):
        out, lse = run_attn(q, pool, opts, lists)
        check_marked(pool, q, out, lse, dtype, lo, hi, opts, range(T))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,rows,group", [(160, 35000, 1024), (40, 70000, 1024), (3, 1 << 20, 4096)],
                         ids=["many", "some", "few"])
def test_attn_every_item_counts(T, rows, group, dtype):
    """Blocks that add a token's rows up in several goes: biases that fall, or rise, with the distance by little enough that
    all of them count; tokens that lie whole in a block, and parts of them, with and without another's output."""
    rng = np.random.default_rng(T)
    pool = MarkedPool(rng, rows, group, dtype, ps=512)
    hi = np.arange(rows - T, rows) + 1
    lo = np.zeros(T, np.int64)
    lists = dict(req=np.zeros(T, np.int32), positions=hi - 1)
    q = flat_queries(rng, T, dtype)
    other = (torch.randn((T, 64, 512), device="cuda") * 0.1).to(DT[dtype]), torch.full((T, 64), float(np.log(rows) - 1), device="cuda")
    tilt = np.float32(rng.uniform(0.1, 1.0, 64) / rows)
    for opts in ({}, dict(slopes=tilt), dict(slopes=-tilt), dict(slopes=-tilt, other=other, sinks=np.float32([5.0] * 64))):
        out, lse = run_attn(q, pool, opts, lists)
        check_marked(pool, q, out, lse, dtype, lo, hi, opts, range(0, T, max(1, T // 20)))


def test_rotate_as_many_tokens_as_an_int_counts():
    """The last of 2^31 - 1 tokens, in place in 34 GB with rows before and behind them."""
    T, D, edge = 2 ** 31 - 1, 8, 64
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("60 GB of device memory are needed")
    buf = torch.zeros((T + 2 * edge, D), dtype=torch.float16, device="cuda")
    buf[:edge], buf[-edge:] = 7.0, 7.0
    x = buf[edge:-edge]
    last = (T - 1) // 65535 * 65535                              # the first token of the last launch
    pick = torch.tensor([0, 1, 65534, 65535, last - 65536, last - 1, last, last + 1, T - 1])
    x[pick.cuda()] = rows = torch.randn((len(pick), D), device="cuda").half()
    pos = torch.arange(T, dtype=I32, device="cuda")
    f = gpu([0.7])
    assert ds4x.rotate(x, pos, f, out=x) is x
    ref = kv16.rotate(rows.double().cpu().numpy(), pick.numpy(), f.cpu().numpy())
    tol = turn_tolerance(ref, rows.double().cpu().numpy(), pick.numpy(), f.cpu().numpy(), "f16")
    assert np.all(np.abs(x[pick.cuda()].double().cpu().numpy() - ref) <= tol)
    assert (buf[:edge] == 7).all() and (buf[-edge:] == 7).all()
    x[pick.cuda()] = 0.0
    assert all(not part.any() for part in x.split(1 << 28))


def test_sizes_beyond_32_bits_are_refused():
    """Tensors whose sizes the library's 32-bit arguments would cut to others that it takes."""
    big = 2 ** 32
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("100 GB of device memory are needed")
    half, f = dict(dtype=torch.float16, device="cuda"), gpu([0.7])
    words = torch.empty(big + 5, dtype=I32, device="cuda")
    for shape in ((big + 5, 8), (1, big + 5, 8), (1, 1, big + 8)):
        with pytest.raises(ValueError, match="too large"):
            ds4x.rotate(torch.empty(shape, **half), words, f)
    many = torch.empty(2 ** 31 + 1, dtype=torch.float64, device="cuda")
    rows, pool = torch.zeros((1, 512), **half), torch.zeros((16, 512), **half)
    one = i32([0])
    with pytest.raises(ValueError, match="too large"):
        ds4x.rotate(rows, one, many)
    with pytest.raises(ValueError, match="too large"):
        ds4x.kv16_append(rows, one, pool, positions=one, inv_freq=many)
    with pytest.raises(ValueError, match="too long"):
        ds4x.kv16_append(torch.empty((1, big + 512), **half), one, pool)
    del many
    q = torch.zeros((1, 64, 512), **half)
    with pytest.raises(ValueError, match="too large"):
        ds4x.kv16_attn(q, pool, words[None, :], one, 1)
    with pytest.raises(ValueError, match="too large"):
        ds4x.kv16_attn(q, pool, words[:, None], words, 16)
    torch.cuda.empty_cache()
