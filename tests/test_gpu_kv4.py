"""The paged 4-bit cache on the GPU against its plain implementation in 64 bits (oracle/kv4.py)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import deepseek_v4_sparse_gb300 as ds4x
from oracle import kv4

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
I32 = torch.int32


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


def rows_of(rng, n, dtype):
    x = rng.standard_normal((n, 512)) * np.exp2(rng.integers(-4, 3, (n, 1)).astype(float))
    return torch.from_numpy(x).to(DT[dtype])


# ------------------------------------------------------------------------------- append and read
def special_rows(dtype):
    """Ties, zeros of both signs, least and largest values, infinities and NaN in groups of their own."""
    x = torch.zeros((6, 512), dtype=torch.float64)
    grid = torch.arange(-32, 33, dtype=torch.float64) / 4               # quarter steps: every tie of e = 0
    x[0, :65], x[0, 96] = grid, 6.0
    x[0, 64:128:2] = -0.0
    for k, e in enumerate((-24, -14, -3, 5, 12)):
        x[1, 64 * k:64 * k + 65] = grid * 2.0 ** e
    x[2] = torch.finfo(DT[dtype]).tiny * torch.linspace(-3, 3, 512, dtype=torch.float64)
    x[3] = torch.finfo(DT[dtype]).max * torch.linspace(-1, 1, 512, dtype=torch.float64)
    x[4, 7], x[4, 40], x[4, 41] = float("inf"), float("-inf"), 1e4
    x[5, 3], x[5, 511], x[5, 510] = float("nan"), float("nan"), float("inf")
    x[5, 100] = 3.0
    return x.to(DT[dtype])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n", [0, 1, 6, 7, 300, 20001])
def test_append_read(n, dtype):
    rng = np.random.default_rng(n)
    x = special_rows(dtype) if n == 6 else rows_of(rng, n, dtype)
    n_slots = n + 11
    slots = rng.permutation(n_slots)[:n].astype(np.int32)
    if n >= 7:
        slots[::5] = -1
        slots[1] = n_slots           # behind the pool
        slots[3] = 2 ** 31 - 1
    codes = rng.integers(0, 256, (n_slots, 256), dtype=np.uint8)
    scales = rng.integers(104, 141, (n_slots, 16), dtype=np.uint8)
    dc, dsc = gpu(codes), gpu(scales)
    ds4x.kv4_append(x.cuda(), i32(slots), dc, dsc)
    m = min(n, 700)                  # the plain form is slow: the first rows bit by bit
    pick = rng.permutation(n)[:m]
    rc, rs = kv4.quantise(x[pick].double().numpy())
    ok = (slots[pick] >= 0) & (slots[pick] < n_slots)
    got_c, got_s = dc.cpu().numpy(), dsc.cpu().numpy()
    at = slots[pick][ok]
    assert np.array_equal(got_s[at], rs[ok])
    codes_count = np.repeat(rs[ok] != 255, 16, axis=1)
    assert np.array_equal(got_c[at][codes_count], rc[ok][codes_count])
    kept = np.setdiff1d(np.arange(n_slots), slots)   # rows of other slots are as they were
    assert np.array_equal(got_c[kept], codes[kept]) and np.array_equal(got_s[kept], scales[kept])
    # read: exact, zeros without a slot, slots may repeat
    again = np.concatenate([slots, slots[:2], [-5]]).astype(np.int32)
    out = ds4x.kv4_read(dc, dsc, i32(again), DT[dtype]).double().cpu().numpy()
    live = (again >= 0) & (again < n_slots)
    ref = np.zeros((len(again), 512))
    ref[live] = kv4.values(got_c[again[live]], got_s[again[live]])
    assert np.array_equal(out, ref, equal_nan=True)


def test_append_takes_slices_of_slots():
    rng = np.random.default_rng(5)
    x = rows_of(rng, 9, "bf16").cuda()
    slots = i32([0, 7, 3, 5, 1, 6, 2, 8, 4])
    pool = torch.zeros((9, 256), dtype=torch.uint8, device="cuda"), torch.zeros((9, 16), dtype=torch.uint8, device="cuda")
    for a, b in ((0, 1), (1, 4), (4, 9)):              # 4-byte aligned starts
        ds4x.kv4_append(x[a:b], slots[a:b], *pool)
    c, s = kv4.quantise(x.double().cpu().numpy())
    assert np.array_equal(pool[0][slots.long()].cpu().numpy(), c)
    assert np.array_equal(pool[1][slots.long()].cpu().numpy(), s)


# ------------------------------------------------------------------------------------- step plan
def plan_case(rng, B, max_pages, ps, ratio, hi_new, spare, T_cap=None, R_cap=None):
    cap = max_pages * ps
    seen = rng.integers(0, cap * ratio + 1, B)
    rows = np.minimum(seen // ratio, cap)
    new = rng.integers(-1, hi_new + 1, B)
    held = -(-rows // ps)
    pages = rng.permutation(int(held.sum()) + max(spare, 1)).astype(np.int32)
    tables = np.full((B, max_pages), -1, dtype=np.int32)
    k = 0
    for b in range(B):
        tables[b, :held[b]] = pages[k:k + held[b]]
        k += held[b]
    T_cap = int(np.maximum(new, 0).sum()) + 3 if T_cap is None else T_cap
    R_cap = int(np.maximum(new, 0).sum()) // ratio + B if R_cap is None else R_cap
    return [seen.astype(np.int32), new.astype(np.int32), rows.astype(np.int32), tables, pages[k:], np.int32(spare),
            ratio, ps, T_cap, R_cap]


def run_plan(c, **kw):
    seen, new, rows, tables, free, n_free, ratio, ps, T_cap, R_cap = c
    dt = i32(tables)
    out = ds4x.page_plan(i32(seen), i32(new), i32(rows), dt, i32(free), i32([n_free]), ratio, ps, T_cap, R_cap, **kw)
    p, r, s, se, ro, nf, to = (x.cpu().numpy() for x in out)
    return p, r, s, dt.cpu().numpy(), se, ro, nf[0], to


def check_plan(got, ref):
    for name, g, r in zip(("positions", "req", "slots", "tables", "seen", "rows", "n_free", "totals"), got, ref):
        assert np.array_equal(g, r), name


@pytest.mark.parametrize("B,max_pages,ps,ratio,hi_new,spare", [
    (1, 1, 1, 1, 1, 1), (1, 5, 8, 4, 1, 3), (3, 4, 16, 1, 40, 2), (64, 9, 64, 4, 1, 64), (65, 3, 8, 3, 200, 30),
    (1000, 6, 4, 7, 60, 4000), (4096, 2, 32, 4, 9, 100), (33, 7, 16, 128, 3000, 0), (1025, 2, 2, 1, 5, 777),
])
def test_page_plan(B, max_pages, ps, ratio, hi_new, spare):
    rng = np.random.default_rng(B * 131 + ps)
    c = plan_case(rng, B, max_pages, ps, ratio, hi_new, spare)
    check_plan(run_plan(c), kv4.page_plan(*c))


@pytest.mark.parametrize("B,max_pages,ps,ratio,hi_new,spare", [
    (1000, 6, 4, 7, 60, 4000), (33, 7, 16, 128, 3000, 0), (5, 40, 64, 4, 5000, 200),
])
def test_page_plan_in_place_over_several_blocks(B, max_pages, ps, ratio, hi_new, spare):
    """The state's outputs are its inputs, with more to fill than one block takes."""
    rng = np.random.default_rng(B + 1)
    c = plan_case(rng, B, max_pages, ps, ratio, hi_new, spare)
    seen, new, rows, tables, free, n_free, ratio, ps, T_cap, R_cap = c
    d = [i32(x) for x in (seen, new, rows, tables, free, [n_free])]
    out = ds4x.page_plan(*d, ratio, ps, T_cap, R_cap, seen_out=d[0], rows_out=d[2], n_free_out=d[5])
    p, r, s, _, _, _, to = (x.cpu().numpy() for x in out)
    got = (p, r, s, d[3].cpu().numpy(), d[0].cpu().numpy(), d[2].cpu().numpy(), d[5].cpu().numpy()[0], to)
    check_plan(got, kv4.page_plan(*c))


def plan_in_a_fresh_process(B):
    """A plan as a process's first call, whose shared memory no earlier call has asked for."""
    c = plan_case(np.random.default_rng(B), B, 2, 8, 4, 9, B)
    check_plan(run_plan(c), kv4.page_plan(*c))


@pytest.mark.parametrize("B", [1732, 1733, 1755, 1756])
def test_page_plan_as_the_first_call(B):
    """28 bytes of shared memory a request, around the 48 KB that a launch has without asking."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = f"from tests.test_gpu_kv4 import plan_in_a_fresh_process as f; f({B})"
    got = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0, got.stderr[-2000:]


def test_page_plan_short_outputs_and_odd_state():
    rng = np.random.default_rng(3)
    c = plan_case(rng, 40, 3, 8, 4, 50, 20, T_cap=100, R_cap=13)          # packed outputs cut off
    check_plan(run_plan(c), kv4.page_plan(*c))
    c[0] = c[0] - 20                                                       # negative seen counts as 0
    c[2] = c[2] * 3 - 10                                                   # rows outside 0 .. cap are clipped
    c[5] = np.int32(10 ** 6)                                               # more free pages than the list holds
    check_plan(run_plan(c), kv4.page_plan(*c))
    c[8], c[9] = 0, 0
    check_plan(run_plan(c), kv4.page_plan(*c))


@pytest.mark.parametrize("spare", [0, 5])
def test_page_plan_without_requests(spare):
    """No tokens, no rows, no pages taken; the free list is as long as before."""
    c = [np.zeros(0, np.int32)] * 3 + [np.zeros((0, 4), np.int32), np.arange(7, dtype=np.int32), np.int32(spare), 4, 8,
                                       0, 0]
    check_plan(run_plan(c, n_free_out=i32([-9]), totals=i32([-9] * 4)), kv4.page_plan(*c))
    check_plan(run_plan(c), kv4.page_plan(*c))
    c[8] = 3
    with pytest.raises(ds4x.Ds4xError):
        run_plan(c)


def test_page_plan_counts_that_pass_32_bits():
    big = 2 ** 31 - 1
    B = 5
    c = [np.array([0, 7, big - 3, big, 100], dtype=np.int32), np.full(B, big, dtype=np.int32),
         np.array([0, 7, 30, 32, 2], dtype=np.int32), np.full((B, 4), -1, dtype=np.int32),
         np.arange(20, dtype=np.int32), np.int32(20), 1, 8, 50, 50]
    check_plan(run_plan(c), kv4.page_plan(*c))
    c[3][:, 0] = 2 ** 30                                                   # a page beyond any slot number
    check_plan(run_plan(c), kv4.page_plan(*c))


def test_page_plan_steps_in_place_and_captured():
    """A decode loop that advances its own state, replayed as a graph."""
    B, ps, ratio, max_pages = 37, 4, 2, 6
    rng = np.random.default_rng(9)
    ref = [np.zeros(B, np.int32), rng.integers(0, 3, B).astype(np.int32), np.zeros(B, np.int32),
           np.full((B, max_pages), -1, np.int32), rng.permutation(150).astype(np.int32), np.int32(150)]
    d = [i32(x) for x in ref[:5]] + [i32([150])]
    T_cap, R_cap = 2 * B, 2 * B
    outs = [torch.empty(n, dtype=I32, device="cuda") for n in (T_cap, T_cap, R_cap)]

    def step():
        return ds4x.page_plan(*d, ratio, ps, T_cap, R_cap, *outs, seen_out=d[0], rows_out=d[2], n_free_out=d[5])
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        totals = step()[-1]
    for i in range(30):
        if i > 0:
            g.replay()
        want = kv4.page_plan(*ref, ratio, ps, T_cap, R_cap)
        got = [x.cpu().numpy() for x in outs] + [d[3].cpu().numpy(), d[0].cpu().numpy(), d[2].cpu().numpy(),
                                                 d[5].cpu().numpy()[0]]
        check_plan(got, want)
        if i > 0:
            assert np.array_equal(totals.cpu().numpy(), want[-1])
        ref[0], ref[2], ref[3], ref[5] = want[4], want[5], want[3], want[6]


# ------------------------------------------------------------------------------------- attention
class Pool:
    """A pool of random rows with every page behind the requests' rows poisoned (NaN groups)."""

    def __init__(self, rng, rows, ps, n_req=None, loud=1.0):
        self.rows, self.ps = np.asarray(rows, dtype=np.int32), ps
        B = len(self.rows)
        held = -(-self.rows // ps)
        self.max_pages = max(1, int(held.max(initial=0)))
        n_pages = int(held.sum()) + 3
        self.n_slots = n_pages * ps
        pages = rng.permutation(n_pages)
        self.tables = np.full((B, self.max_pages), -1, dtype=np.int32)
        self.codes = rng.integers(0, 256, (self.n_slots, 256), dtype=np.uint8)
        self.scales = np.full((self.n_slots, 16), 255, dtype=np.uint8)     # what nobody holds reads as NaN
        k = 0
        for b in range(B):
            self.tables[b, :held[b]] = pages[k:k + held[b]]
            k += held[b]
            for pg in range(held[b]):
                n = min(ps, self.rows[b] - pg * ps)
                at = self.tables[b, pg] * ps
                self.scales[at:at + n] = rng.integers(124, 127, (n, 16)) if loud == 1.0 else \
                    rng.integers(127, 131, (n, 16))
        self.dev = gpu(self.codes), gpu(self.scales), i32(self.tables), i32(self.rows)

    def values(self):
        return kv4.values(self.codes, self.scales)


def tolerance(q, kv, out, scale, dtype):
    """How far out [64, 512] and lse [64] of one token over rows kv [n, 512] may be.

    Logits: 512 exact products summed in fp32; each of the sum's steps is off by at most 2^-23 (a
    truncating adder) of the sum of magnitudes, and the 32 matrix steps add 16 products each; with the
    products' own inner sums 64 steps cover it: ex = 64 * 2^-23 * scale * sum |q||kv|, plus 2^-20 for
    2^x and its argument (2^-22 and |x| 2^-24 with |x| < 100).
    Weights: 2 ex relative, and rounded to 16 bits (half a step of fp16, 2^-11) once, in numerator and
    normaliser alike: a normalised weight moves by at most eta = 2 (2^-11 + 2 ex) relative, and
    |out - ref| <= eta * sum_j w_j |kv_j - ref|.  Weights below fp16's normal range (the largest is at
    least 2^-8 times 2^7) are off by 2^-25 absolutely, n of them against a sum of at least 2^-1.
    The output is rounded once: half a step of its type, 2^-25 below fp16's normal range."""
    x = (q @ kv.T) * scale
    ex = 64 * 2.0 ** -23 * scale * (np.abs(q) @ np.abs(kv).T).max(axis=1) + 2.0 ** -20
    w = np.exp(x - x.max(axis=1, keepdims=True))
    w /= w.sum(axis=1, keepdims=True)
    spread = np.stack([w[h] @ np.abs(kv - out[h][None, :]) for h in range(q.shape[0])])
    eta = 2 * (2.0 ** -11 + 2 * ex)
    half = torch.finfo(DT[dtype]).eps / 2
    tiny = kv.shape[0] * 2.0 ** -24 * np.abs(kv).max()
    return (eta[:, None] * spread + tiny + half * np.abs(out) * 1.01 + 2.0 ** -25,
            2 * ex + 2.0 ** -20 * (1 + np.abs(x).max(axis=1)))


def check_attn(q, pool, got, lse, scale, dtype, lists):
    vals = pool.values()
    qd = q.double().cpu().numpy()
    tabs = dict(tables=pool.tables, rows=pool.rows, page_rows=pool.ps)
    ref, rlse = kv4.attn(qd, vals, scale, **tabs, **lists)
    g, gl = got.double().cpu().numpy(), lse.double().cpu().numpy()
    for t in range(q.shape[0]):
        at = kv4.attended_slots(t, n_slots=pool.n_slots, **tabs, **lists)
        if not at:
            assert np.all(g[t] == 0) and np.all(np.isneginf(gl[t])), t
            continue
        tol, ltol = tolerance(qd[t], vals[at], ref[t], scale, dtype)
        assert np.all(np.isfinite(g[t])), t
        worst = (np.abs(g[t] - ref[t]) / tol).max()
        assert worst <= 1, (t, len(at), worst)
        assert np.all(np.abs(gl[t] - rlse[t]) <= ltol), (t, np.abs(gl[t] - rlse[t]).max())


def queries(rng, T, dtype, size=1.0):
    return torch.from_numpy(rng.standard_normal((T, 64, 512)) * size).to(DT[dtype]).cuda()


def run_attn(q, pool, scale=None, **lists):
    kw = {k: (v if k == "ratio" or v is None else i32(v)) for k, v in lists.items()}
    return ds4x.kv4_attn(q, *pool.dev, pool.ps, scale=scale, **kw)


SCALE = 512 ** -0.5


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,rows,ps,k_top", [
    (1, [700], 64, 512), (1, [40], 8, 512), (3, [65, 1, 200], 16, 64), (7, [1000] * 7, 32, 333),
    (5, [64, 63, 65, 128, 0], 1, 100), (2, [2000, 1500], 256, 1024), (150, [300] * 150, 64, 70), (1, [1], 128, 1),
])
def test_attn_selected(T, rows, ps, k_top, dtype):
    rng = np.random.default_rng(T * 7 + k_top)
    pool = Pool(rng, rows, ps)
    idx = np.full((T, k_top), -1, dtype=np.int32)
    counts = np.zeros(T, dtype=np.int32)
    for t in range(T):
        n = min(k_top, rows[t])
        idx[t, :n] = np.sort(rng.permutation(rows[t])[:n])
        counts[t] = n
    q = queries(rng, T, dtype)
    for lists in (dict(indices=idx), dict(indices=idx, counts=counts)):
        out, lse = run_attn(q, pool, **lists)
        check_attn(q, pool, out, lse, SCALE, dtype, lists)


def test_attn_selected_odd_lists():
    """Lists with holes, repeats, rows that are not held, and rows without a page; a request that is none."""
    rng = np.random.default_rng(4)
    pool = Pool(rng, [150, 90, 30, 1], 16)
    pool.tables[1, 2] = -7                                     # rows 32..47 of request 1 have no page
    pool.tables[2, 0] = pool.n_slots // 16                     # rows 0..15 of request 2 are behind the pool
    pool.tables[3, 0] = 2 ** 31 - 1
    pool.dev = *pool.dev[:2], i32(pool.tables), pool.dev[3]
    req = np.array([1, 0, 2, 0, -1, 4, 3, 1, 2 ** 31 - 1], dtype=np.int32)
    T = len(req)
    idx = rng.integers(-40, 200, (T, 200)).astype(np.int32)
    idx[1] = 149                                               # one row, 200 times
    idx[3] = -1
    idx[7, :] = 2 ** 31 - 1
    counts = np.array([200, 199, 65, 64, 200, 10, 200, -3, 0], dtype=np.int32)
    q = queries(rng, T, "bf16")
    for lists in (dict(req=req, indices=idx), dict(req=req, indices=idx, counts=counts),
                  dict(req=req, indices=idx, counts=counts * 1000)):
        out, lse = run_attn(q, pool, **lists)
        check_attn(q, pool, out, lse, SCALE, "bf16", lists)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,ps,req,ratio,back", [
    ([1], 64, [0], 1, 0), ([64], 16, [0], 4, 0), ([65], 16, [0], 4, 0), ([5000], 64, [0], 128, 0),
    ([0, 3, 127, 128, 129, 700], 32, [0, 1, 2, 3, 4, 5], 128, 0),
    ([300, 77], 8, [0] * 20 + [1] * 13, 4, 37), ([40], 1, [0] * 170, 1, 169),
    ([2500, 10, 900], 128, [2, 0, 1, 0, 2], 7, 3),
])
def test_attn_all_visible(rows, ps, req, ratio, back, dtype):
    rng = np.random.default_rng(len(req) * 11 + ps)
    pool = Pool(rng, rows, ps)
    req = np.array(req, dtype=np.int32)
    # positions up to the last one; the first tokens may see nothing, or be before the sequence
    positions = (np.array(rows)[req] * ratio - 1 - rng.integers(0, back + 1, len(req)) * max(1, ratio // 2)).astype(np.int32)
    q = queries(rng, len(req), dtype)
    for lists in (dict(req=req, positions=positions, ratio=ratio), dict(req=req)):
        out, lse = run_attn(q, pool, **lists)
        check_attn(q, pool, out, lse, SCALE, dtype, lists)


def test_attn_request_of_a_token_is_its_number():
    rng = np.random.default_rng(12)
    pool = Pool(rng, [10, 200, 64], 64)
    q = queries(rng, 2, "f16")
    out, lse = run_attn(q, pool)
    check_attn(q, pool, out, lse, SCALE, "f16", {})
    none = Pool(rng, [0, 0], 8)
    out, lse = run_attn(q, none)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size,loud", [(1e-4, 1.0), (30.0, 1.0), (1.0, 8.0), (60.0, 8.0)])
def test_attn_small_and_large_logits(size, loud, dtype):
    """Uniform weights, and one row that takes all: the running maximum has to move, late rows included."""
    rng = np.random.default_rng(int(size * 10))
    pool = Pool(rng, [900, 333], 32, loud=loud)
    q = queries(rng, 2, dtype, size)
    q[0, 0] = 0
    q[0, 1, 1:] = 0
    # the row with the largest logit of some heads comes last
    q[1, 5] = torch.from_numpy(pool.values()[kv4.attended_slots(1, pool.tables, pool.rows, 32, pool.n_slots)[-1]]).to(DT[dtype])
    lists = dict(req=np.array([0, 1], dtype=np.int32))
    out, lse = run_attn(q, pool, **lists)
    check_attn(q, pool, out, lse, SCALE, dtype, lists)


def test_attn_extreme_queries():
    """bf16 queries beyond fp16's range, heads of very different sizes."""
    rng = np.random.default_rng(77)
    pool = Pool(rng, [130, 64], 16)
    q = queries(rng, 2, "bf16")
    for h, e in enumerate(range(-100, 100, 4)):
        q[:, h] *= 2.0 ** e
    q[0, 50], q[1, 51, ::2] = 0, 2.0 ** -126
    for scale in (SCALE, 2.0 ** -96, -0.02):
        lists = dict(req=np.array([0, 1], dtype=np.int32))
        out, lse = run_attn(q, pool, scale=scale, **lists)
        qd, vals = q.double().cpu().numpy(), pool.values()
        tabs = dict(tables=pool.tables, rows=pool.rows, page_rows=16)
        ref, rlse = kv4.attn(qd, vals, scale, **tabs, **lists)
        for t in range(2):
            at = kv4.attended_slots(t, n_slots=pool.n_slots, **tabs, **lists)
            x = (qd[t] @ vals[at].T) * scale
            size = abs(scale) * (np.abs(qd[t]) @ np.abs(vals[at]).T).max(axis=1)
            calm = size < 2000                 # beyond, fp32 logits do not decide between near rows
            tol, ltol = tolerance(qd[t], vals[at], ref[t], abs(scale), "bf16")
            g = out[t].double().cpu().numpy()
            assert np.all(np.abs(g - ref[t])[calm] <= tol[calm])
            assert np.all(np.abs(lse[t].double().cpu().numpy() - rlse[t])[calm] <= ltol[calm])
            assert np.isfinite(g[np.abs(x).max(axis=1) < 1e30]).all()


def test_attn_nan_rows_reach_only_those_who_attend():
    rng = np.random.default_rng(31)
    pool = Pool(rng, [100, 100], 16)
    bad = int(pool.tables[0, 2]) * 16 + 5                     # row 37 of request 0
    pool.scales[bad, 3] = 255
    pool.dev = pool.dev[0], gpu(pool.scales), *pool.dev[2:]
    q = queries(rng, 3, "f16")
    idx = np.stack([np.arange(100), np.arange(100), np.arange(100)]).astype(np.int32)
    idx[1, 37] = -1
    req = np.array([0, 0, 1], dtype=np.int32)
    out, lse = run_attn(q, pool, req=req, indices=idx)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert torch.isfinite(out[1:]).all() and torch.isfinite(lse[1:]).all()


def test_attn_outputs_streams_and_neighbours():
    """Into slices of larger buffers, on another stream, without lse; what lies around stays."""
    rng = np.random.default_rng(6)
    pool = Pool(rng, [500, 70, 9], 32)
    req = np.array([0, 2, 1, 0, 1], dtype=np.int32)
    q = queries(rng, 5, "bf16")
    want, wlse = run_attn(q, pool, req=req)
    big = torch.full((9, 64, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    blse = torch.full((9, 64), 3.0, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ds4x.kv4_attn(q, *pool.dev, 32, req=i32(req), out=big[2:7], lse=blse[2:7], stream=s)
    only, none = ds4x.kv4_attn(q, *pool.dev, 32, req=i32(req), want_lse=False, stream=s.cuda_stream)
    s.synchronize()
    assert none is None and torch.equal(only, want)
    assert torch.equal(big[2:7], want) and torch.equal(blse[2:7], wlse)
    assert (big[:2] == 3).all() and (big[7:] == 3).all() and (blse[:2] == 3).all() and (blse[7:] == 3).all()


def test_attn_two_graphs_share_a_workspace():
    rng = np.random.default_rng(8)
    pool = Pool(rng, [3000, 40, 600], 64)
    need = ds4x.kv4_attn_workspace_bytes(6, pool.max_pages * 64)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")   # nothing is read before it is written
    cases = []
    for req in ([0], [1, 2, 0, 0, 2, 1]):
        q, r = queries(rng, len(req), "f16"), i32(req)
        want = ds4x.kv4_attn(q, *pool.dev, 64, req=r)
        out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ds4x.kv4_attn(q, *pool.dev, 64, req=r, out=out, lse=lse, workspace=ws)
        cases.append((g, q, r, want, out, lse))
    for k in (0, 1, 1, 0, 1):
        g, _, _, want, out, lse = cases[k]
        out.zero_(), lse.zero_()
        g.replay()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_attn_is_the_same_twice_and_per_token():
    """Same bits on every run; a token's result is near that of the token alone."""
    rng = np.random.default_rng(13)
    pool = Pool(rng, rng.integers(1, 1500, 40), 32)
    req = rng.integers(0, 40, 333).astype(np.int32)
    q = queries(rng, 333, "f16")
    out, lse = run_attn(q, pool, req=req)
    for _ in range(3):
        o2, l2 = run_attn(q, pool, req=req)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    for t in (0, 100, 332):
        o1, l1 = run_attn(q[t:t + 1].clone(), pool, req=req[t:t + 1])
        # two results within the tolerance each; unit-size values, far from it in practice
        assert (o1[0].float() - out[t].float()).abs().max() < 4e-3
        assert (l1[0] - lse[t]).abs().max() < 1e-4


def test_attn_many_tokens():
    """More tokens than one launch plans for; sampled against the plain form."""
    rng = np.random.default_rng(21)
    pool = Pool(rng, rng.integers(0, 90, 50), 16)
    T = 5003
    req = rng.integers(-1, 51, T).astype(np.int32)
    q = queries(rng, 64, "bf16").repeat((T + 63) // 64, 1, 1)[:T].contiguous()
    out, lse = run_attn(q, pool, req=req)
    some = np.unique(np.concatenate([rng.integers(0, T, 40), [0, 2047, 2048, 2049, 4095, 4096, T - 1]]))
    check_attn(q[some], pool, out[some], lse[some], SCALE, "bf16", dict(req=req[some]))


def test_attn_without_any_rows():
    """Tables without pages, a pool without slots, no requests at all: zeros and -inf, nothing is read."""
    q = queries(np.random.default_rng(1), 3, "f16")
    none = torch.zeros((0, 256), dtype=torch.uint8, device="cuda"), torch.zeros((0, 16), dtype=torch.uint8, device="cuda")
    pool = torch.zeros((64, 256), dtype=torch.uint8, device="cuda"), torch.full((64, 16), 255, dtype=torch.uint8, device="cuda")
    idx = i32(np.arange(200)[None].repeat(3, 0))
    cases = [
        (pool, i32(np.zeros((3, 0))), i32([5, 9, 64]), dict()),                      # no page fits a table
        (pool, i32(np.zeros((3, 0))), i32([5, 9, 64]), dict(indices=idx)),
        (none, i32([[0], [0], [0]]), i32([5, 9, 64]), dict()),                       # no slot in the pool
        (none, i32([[0], [0], [0]]), i32([5, 9, 64]), dict(indices=idx)),
        (pool, i32(np.zeros((0, 2))), i32([]), dict(req=i32([0, 1, -1]))),           # no requests
        (pool, i32(np.zeros((0, 2))), i32([]), dict(req=i32([0, 1, -1]), indices=idx)),
        (pool, i32([[0], [0], [0]]), i32([0, -4, 0]), dict(indices=idx)),            # nothing held
    ]
    for (codes, scales), tables, rows, lists in cases:
        out, lse = ds4x.kv4_attn(q, codes, scales, tables, rows, 64, out=torch.full_like(q, 7.0), **lists)
        assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
    empty, _ = ds4x.kv4_attn(q[:0], *pool, i32([[0]]), i32([1]), 64)
    assert empty.shape == (0, 64, 512)


@pytest.mark.parametrize("T", [2049, 4100])
def test_attn_a_few_tokens_behind_a_full_launch(T):
    """The last launch has few tokens, with long lists split over every block."""
    rng = np.random.default_rng(T)
    pool = Pool(rng, [9, 3000], 64)
    req = np.zeros(T, dtype=np.int32)
    req[2048:2049] = req[T - 1:] = 1
    q = queries(rng, 16, "f16").repeat((T + 15) // 16, 1, 1)[:T].contiguous()
    out, lse = run_attn(q, pool, req=req)
    some = np.array([0, 2047, 2048, T - 1])
    check_attn(q[some], pool, out[some], lse[some], SCALE, "f16", dict(req=req[some]))


@pytest.mark.parametrize("rows", [65536, 4194304])
def test_attn_long_lists_in_one_block(rows):
    """A token for every SM, each over the same page again and again: every block has one long item.

    Attention over n copies of 64 rows is attention over the 64 rows, and ln(n) more in lse.  The products add
    16 rows to fp32 sums at a time, each step off by at most 2^-23 of the sum of magnitudes (a truncating adder):
    rows / 16 * 2^-23 of sum_j w_j |kv_j|, beside what tolerance() counts for the 64 rows.  The sums of the
    weights round each of their (rows / 8 a thread) steps by 2^-24."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rng = np.random.default_rng(5)
    codes = rng.integers(0, 256, (64, 256), dtype=np.uint8)
    scales = rng.integers(124, 127, (64, 16)).astype(np.uint8)
    q = queries(rng, sms, "f16")
    out, lse = ds4x.kv4_attn(q, gpu(codes), gpu(scales), torch.zeros((1, rows // 64), dtype=I32, device="cuda"),
                             i32([rows]), 64, req=torch.zeros(sms, dtype=I32, device="cuda"))
    assert ds4x.device_status() == ds4x.OK
    vals, scale = kv4.values(codes, scales), 1 / np.sqrt(512)
    once = dict(tables=np.zeros((1, 1), np.int32), rows=[64], page_rows=64, req=np.zeros(1, np.int32))
    for t in (0, sms - 1):
        qd = q[t:t + 1].double().cpu().numpy()
        ref, rlse = kv4.attn(qd, vals, scale, **once)
        tol, ltol = tolerance(qd[0], vals, ref[0], scale, "f16")
        x = (qd[0] @ vals.T) * scale
        w = np.exp(x - rlse[0][:, None])
        steps = rows / 16 * 2.0 ** -23
        grow = steps * (w @ np.abs(vals)) + rows / 8 * 2.0 ** -24 * np.abs(ref[0])
        assert np.all(np.abs(out[t].double().cpu().numpy() - ref[0]) <= tol + grow)
        assert np.all(np.abs(lse[t].double().cpu().numpy() - rlse[0] - np.log(rows / 64)) <=
                      ltol + rows / 8 * 2.0 ** -24 + 2.0 ** -20)


def test_attn_two_calls_at_once():
    """On two streams, each with its own workspace, many times over."""
    rng = np.random.default_rng(50)
    pool = Pool(rng, [2500, 700, 60], 32)
    req = [np.array([0, 1, 2, 0], dtype=np.int32), rng.integers(0, 3, 300).astype(np.int32)]
    qs = [queries(rng, len(r), "bf16") for r in req]
    want = [run_attn(q, pool, req=r) for q, r in zip(qs, req)]
    dr = [i32(r) for r in req]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for k in (0, 1):
            got[k].append(ds4x.kv4_attn(qs[k], *pool.dev, 32, req=dr[k], stream=streams[k]))
    torch.cuda.synchronize()
    for k in (0, 1):
        for out, lse in got[k]:
            assert torch.equal(out, want[k][0]) and torch.equal(lse, want[k][1])


def test_binding_refuses_on_the_device():
    rng = np.random.default_rng(2)
    pool = Pool(rng, [20, 30], 16)
    q = queries(rng, 2, "f16")
    codes, scales, tables, rows = pool.dev

    def bad(match, *a, **kw):
        with pytest.raises(ValueError, match=match):
            ds4x.kv4_attn(*a, **kw)
    bad("contiguous", q.transpose(0, 1).contiguous().transpose(0, 1), *pool.dev, 16)
    bad("contiguous", q, codes, scales, tables.t().contiguous().t(), rows, 16) if tables.shape[1] > 1 else None
    bad("slots", q, codes, scales[:-1], tables, rows, 16)
    bad("256", q, codes[:, :128].contiguous(), scales, tables, rows, 16)
    bad("int32", q, codes, scales, tables.long(), rows, 16)
    bad("max_pages", q, codes, scales, tables[:1], rows, 16)
    bad("CUDA", q, codes, scales, tables, rows.cpu(), 16)
    bad("counts belong", q, *pool.dev, 16, counts=rows)
    bad("indices must be", q, *pool.dev, 16, indices=i32(np.zeros((3, 8))))
    bad("holds 1", q, *pool.dev, 16, req=i32([0]))
    bad("shape", q, *pool.dev, 16, out=torch.empty_like(q[:1]))
    bad("shape", q, *pool.dev, 16, lse=torch.empty((2, 32), device="cuda"))
    bad("float16 or bfloat16", q.float(), *pool.dev, 16)
    for kw, status in ((dict(page_rows=24), ds4x.ERR_UNSUPPORTED), (dict(page_rows=0), ds4x.ERR_INVALID)):
        with pytest.raises(ds4x.Ds4xError) as e:
            ds4x.kv4_attn(q, *pool.dev, **kw)
        assert e.value.status == status
    with pytest.raises(ds4x.Ds4xError) as e:                       # three tokens, two requests
        ds4x.kv4_attn(queries(rng, 3, "f16"), *pool.dev, 16)
    assert e.value.status == ds4x.ERR_INVALID
    with pytest.raises(ds4x.Ds4xError) as e:
        ds4x.kv4_attn(q, *pool.dev, 16, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == ds4x.ERR_WORKSPACE
    with pytest.raises(ValueError, match="must not be negative"):
        ds4x.page_plan(rows, rows, rows, tables, rows, rows[:1], 4, 16, -1, 5)
    with pytest.raises(ValueError, match="holds 1"):
        ds4x.kv4_append(torch.zeros((2, 512), dtype=torch.float16, device="cuda"), i32([0]), codes, scales)
    with pytest.raises(ds4x.Ds4xError):                            # rows of another width
        ds4x.kv4_append(torch.zeros((2, 128), dtype=torch.float16, device="cuda"), i32([0, 1]), codes, scales)


# ------------------------------------------------------------------------------ a run of them all
def test_serving_steps_end_to_end():
    """Steps of a batch as a server runs them: plan, compress, append, score and top-k, attention; the
    16-bit path over the rows read back gives the same."""
    rng = np.random.default_rng(40)
    B, ratio, ps, max_pages, k_top = 3, 4, 16, 12, 24
    lens = [(50, 300, 7), (1, 1, 1), (3, 0, 200), (1, 1, 1)]
    dev = "cuda"
    seen, rows = i32([0] * B), i32([0] * B)
    tables, free, n_free = i32(np.full((B, max_pages), -1)), i32(rng.permutation(40)), i32([40])
    pool = (torch.zeros((40, ps, 256), dtype=torch.uint8, device=dev), torch.zeros((40, ps, 16), dtype=torch.uint8, device=dev))
    k_rows = [torch.zeros((max_pages * ps, 128), dtype=torch.float16, device=dev) for _ in range(B)]
    frontier = [(None, None)] * B
    kv_all = [[] for _ in range(B)]
    bias = torch.zeros((ratio, 512), device=dev)
    for new in lens:
        T = sum(new)
        R_cap = T // ratio + B
        before = rows.cpu().tolist()
        positions, req, slots, seen, rows, n_free, totals = ds4x.page_plan(
            seen, i32(new), rows, tables, free, n_free, ratio, ps, T, R_cap)
        at = 0
        for b in range(B):
            x, g = (torch.from_numpy(rng.standard_normal((new[b], 512))).to(torch.bfloat16).cuda() for _ in range(2))
            out, fx, fg = ds4x.compress(x, g, bias, ratio, *frontier[b]) if new[b] else (x, *frontier[b])
            frontier[b] = (fx, fg) if fx is not None and fx.shape[0] else (None, None)
            n = out.shape[0]
            ds4x.kv4_append(out, slots[at:at + n], *pool)
            k_rows[b][before[b]:before[b] + n] = torch.from_numpy(rng.standard_normal((n, 128))).half().cuda()
            kv_all[b].append(out)
            at += n
        held = rows.cpu().tolist()
        assert totals.cpu().tolist()[:3] == [T, at, at]
        q = queries(rng, T, "bf16")
        qi = torch.from_numpy(rng.standard_normal((T, 16, 128))).half().cuda()
        w = torch.from_numpy(rng.random((T, 16))).half().cuda()
        idx = torch.empty((T, k_top), dtype=I32, device=dev)
        counts = torch.empty((T,), dtype=I32, device=dev)
        t0 = 0
        for b in range(B):                                   # scores and top-k of each request's tokens
            if new[b] == 0:
                continue
            sl = slice(t0, t0 + new[b])
            S = max(1, held[b])
            p = positions[sl].clone()
            sc = ds4x.indexer_score(qi[sl].clone(), w[sl].clone(), k_rows[b], p, ratio, S=S)
            i, c = ds4x.topk(sc, p, min(S, held[b]) if held[b] else 0, ratio, k_top) if held[b] else \
                (torch.full((new[b], k_top), -1, dtype=I32, device=dev), torch.zeros(new[b], dtype=I32, device=dev))
            idx[sl], counts[sl] = i, c
            t0 += new[b]
        for lists in (dict(indices=idx, counts=counts), dict(positions=positions, ratio=ratio)):
            out, lse = ds4x.kv4_attn(q, *pool, tables, rows, ps, req=req, **lists)
            t0 = 0
            for b in range(B):
                if new[b] == 0:
                    continue
                r = torch.arange(max(1, held[b]), device=dev)
                own = tables[b][r // ps] * ps + r.int() % ps
                kv = ds4x.kv4_read(*pool, own.int(), torch.bfloat16)
                if held[b]:
                    c, s = kv4.quantise(torch.cat(kv_all[b]).double().cpu().numpy())
                    assert np.array_equal(kv.double().cpu().numpy(), kv4.values(c, s))
                sl = slice(t0, t0 + new[b])
                if "indices" in lists:
                    i16 = idx[sl].clone()
                else:
                    n = (positions[sl] + 1) // ratio
                    i16 = torch.where(torch.arange(192, device=dev)[None, :] < n[:, None], torch.arange(192, device=dev)[None, :], -1).int()
                ref, rlse = ds4x.sparse_attn(q[sl].clone(), kv, i16, S=held[b])
                # the 16-bit path rounds its weights to bf16 (2^-8, values below 6): 2 * 2^-8 * 6
                assert (out[sl].float() - ref.float()).abs().max() <= 0.05
                fin = torch.isfinite(rlse)
                assert torch.equal(fin, torch.isfinite(lse[sl]))
                assert (lse[sl][fin] - rlse[fin]).abs().max() <= 2.0 ** -7 if fin.any() else True
                t0 += new[b]


@pytest.mark.parametrize("given", ["nothing", "workspace", "counts", "many tokens"])
def test_attn_lists_of_width_zero(given):
    """An index list without entries names no row, whatever the requests hold."""
    rng = np.random.default_rng(60)
    pool = Pool(rng, [300, 0, 65], 16)
    T = 2051 if given == "many tokens" else 3
    req = rng.integers(0, 3, T).astype(np.int32)
    q = queries(rng, 3, "bf16").repeat((T + 2) // 3, 1, 1)[:T].contiguous()
    kw = dict(req=i32(req), positions=i32(np.full(T, 10 ** 6)))
    if given == "workspace":
        kw["workspace"] = torch.empty(ds4x.kv4_attn_workspace_bytes(T, pool.max_pages * 16), dtype=torch.uint8, device="cuda")
    if given == "counts":
        kw["counts"] = i32([5, 0, -1])
    wide = i32(np.zeros((T, 8)))
    for idx in (torch.empty((T, 0), dtype=I32, device="cuda"), wide[:, :0].contiguous(), wide[:, :0]):
        out, lse = ds4x.kv4_attn(q, *pool.dev, 16, indices=idx, out=torch.full_like(q, 7.0), **kw)
        assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
    with pytest.raises(ValueError, match="indices must be"):
        ds4x.kv4_attn(q, *pool.dev, 16, indices=torch.empty((T + 1, 0), dtype=I32, device="cuda"), **kw)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("ratio", [1, 4])
def test_a_request_that_ran_short_keeps_its_rows_in_order(ratio, in_place):
    """Steps of which one finds too few pages: row r of a request is its r-th pooled row in every step, so a
    token attends to pooled rows before it only; what has no place is missing, and rows_out says so."""
    rng = np.random.default_rng(61)
    B, ps, max_pages, pages = 3, 4, 12, 20
    start, free_after = [40, 9, 0], [3, 12, 0]                # pages that come back before each later step
    steps = [np.array(n) * ratio for n in ([10, 6, 5], [7, 7, 3], [5, 1, 9])]
    truth = rng.standard_normal((B, 100, 512))                # pooled row r of request b
    truth[:, :, 0] = np.arange(100)[None] / 4                 # tells the rows apart
    truth = torch.from_numpy(truth).half()
    seen, rows = np.array(start) // 4 * ratio, np.array(start) // 4
    held = -(-rows // ps)
    tables = np.full((B, max_pages), -1)
    order = rng.permutation(pages)
    for b in range(B):
        tables[b, :held[b]] = order[sum(held[:b]):sum(held[:b + 1])]
    free = list(order[sum(held):])
    pool = torch.zeros((pages, ps, 256), dtype=torch.uint8, device="cuda"), torch.zeros((pages, ps, 16), dtype=torch.uint8, device="cuda")
    for b in range(B):
        r = np.arange(rows[b])
        if len(r):
            ds4x.kv4_append(truth[b, :rows[b]].cuda(), i32(tables[b][r // ps] * ps + r % ps), *pool)
    values = [kv4.values(*kv4.quantise(truth[b].double().numpy())) for b in range(B)]
    dseen, drows, dtables = i32(seen), i32(rows), i32(tables)
    n_free = 4                                                # of the list's pages, at the first step
    short = np.zeros(B, dtype=bool)
    for new, back in zip(steps, free_after):
        T, R = int(new.sum()), int(new.sum()) // ratio + B
        kw = {}
        dfree, dn = i32(free if free else [0]), i32([min(n_free, len(free))])
        if in_place:
            kw = dict(seen_out=dseen, rows_out=drows, n_free_out=dn)
        positions, req, slots, dseen, drows, dn, totals = ds4x.page_plan(
            dseen, i32(new), drows, dtables, dfree, dn, ratio, ps, T, R, **kw)
        first = seen // ratio
        seen = seen + new
        done = seen // ratio - first
        x = torch.cat([truth[b, first[b]:first[b] + done[b]] for b in range(B)]).cuda()
        ds4x.kv4_append(x, slots, *pool)                      # the rows that the step completed, in its order
        assert np.array_equal(dseen.cpu().numpy(), seen)
        now = drows.cpu().numpy()
        assert np.all(now[short] == rows[short])              # nothing is added behind a gap
        rows, short = now, now < seen // ratio
        left = int(dn.cpu()[0])
        assert totals.cpu().tolist()[3] == min(n_free, len(free)) - left
        free = free[:left] + free[min(n_free, len(free)):]
        n_free = left + back
        q = queries(rng, T, "f16")
        out, lse = ds4x.kv4_attn(q, *pool, dtables, drows, ps, req=req, positions=positions, ratio=ratio)
        for t in range(T):
            b, pos = int(req[t]), int(positions[t])
            n = min(int(rows[b]), (pos + 1) // ratio)
            if n == 0:
                assert torch.all(out[t] == 0)
                continue
            kv = values[b][:n]
            qd = q[t].double().cpu().numpy()
            x = (qd @ kv.T) * SCALE
            w = np.exp(x - x.max(axis=1, keepdims=True))
            ref = w @ kv / w.sum(axis=1, keepdims=True)
            tol, _ = tolerance(qd, kv, ref, SCALE, "f16")
            assert np.all(np.abs(out[t].double().cpu().numpy() - ref) <= tol), (b, pos)
    assert short.any()


def test_attn_sums_of_very_long_lists_are_not_biased():
    """4194304 rows of one token in a block.  Dims 32.. are the same in every row, so out is that value: what
    is left is the error of the sums alone (the weights' rounding stands in numerator and normaliser alike).

    A list is added up 16384 rows at a time.  O^T: 1024 steps of 16 products, each of which the matrix unit may
    add in four truncating parts, so each is off by less than 2^-21 of the sum so far, half of that over a chain
    of growing sums: 1024 / 2 * 2^-21 = 2^-12.  The normaliser: 4096 terms a thread, each step rounded by 2^-24
    of the sum so far, half of that: 2^-13.  The 256 sums are joined by two products and an addition each:
    256 * 3 / 2 * 2^-24, in numerator and normaliser.  The output is rounded once: 2^-11 relative.  lse: as the
    normaliser, the factors of 2^x at 2^-22 a join, and the logits' part of tolerance()."""
    rows = 4194304
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rng = np.random.default_rng(63)
    codes = np.tile(rng.integers(1, 8, (1, 256), dtype=np.uint8) * 17, (64, 1))   # both nibbles: positive values
    codes[:, :16] = rng.integers(0, 256, (64, 16), dtype=np.uint8)                # dims 0..31: the logits
    scales = np.full((64, 16), 127, dtype=np.uint8)
    q = queries(rng, sms, "f16")
    q[:, :, 32:] = 0
    out, lse = ds4x.kv4_attn(q, gpu(codes), gpu(scales), torch.zeros((1, rows // 64), dtype=I32, device="cuda"),
                             i32([rows]), 64, req=torch.zeros(sms, dtype=I32, device="cuda"))
    assert ds4x.device_status() == ds4x.OK
    vals = kv4.values(codes, scales)
    norm = 2.0 ** -13 + 256 * 3 / 2 * 2.0 ** -24
    for t in (0, 1, sms - 1):
        qd = q[t].double().cpu().numpy()
        want = vals[0, 32:]
        got = out[t, :, 32:].double().cpu().numpy()
        worst = np.abs(got / want - 1).max()
        assert worst <= 2.0 ** -12 + 256 * 3 / 2 * 2.0 ** -24 + norm + 2.0 ** -11, worst
        x = (qd @ vals.T) * SCALE
        m = x.max(axis=1, keepdims=True)
        rlse = m[:, 0] + np.log(np.exp(x - m).sum(axis=1)) + np.log(rows / 64)
        ref = np.exp(x - m) @ vals / np.exp(x - m).sum(axis=1, keepdims=True)
        _, ltol = tolerance(qd, vals, ref, SCALE, "f16")
        assert np.all(np.abs(lse[t].double().cpu().numpy() - rlse) <= ltol + norm + 256 * 2.0 ** -22)


@pytest.mark.parametrize("dtype,size", [("f16", 1.0), ("bf16", 30.0)])
def test_attn_long_lists_added_up_in_parts(dtype, size):
    """Tokens of several times 16384 rows a block, whole in a block or over two, among short ones; the largest
    logits come late."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rng = np.random.default_rng(64)
    pool = Pool(rng, [20000, 70000, 3, 0], 64)
    late = pool.tables[1, -3:, None] * 64 + np.arange(40)
    pool.scales[late[late < pool.n_slots].ravel()] += 2
    pool.dev = pool.dev[0], gpu(pool.scales), *pool.dev[2:]
    req = np.concatenate([[2, 1, 3, 0], rng.choice([0, 1, 1, 1, 2, 3], 3 * sms // 2), [1, 0]]).astype(np.int32)
    T = len(req)
    # visible rows: a few short of all, so that tokens start and end at different places of the blocks
    positions = (pool.rows[req] - 1 - rng.integers(0, 300, T)).astype(np.int32)
    q = queries(rng, T, dtype, size)
    out, lse = run_attn(q, pool, req=req, positions=positions, ratio=1)
    assert torch.isfinite(out).all()
    o2, l2 = run_attn(q, pool, req=req, positions=positions, ratio=1)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    vals = torch.from_numpy(pool.values()).cuda()
    for t in np.unique(np.concatenate([np.arange(4), [T - 2, T - 1], rng.integers(0, T, 20)])):
        at = kv4.attended_slots(t, pool.tables, pool.rows, 64, pool.n_slots, req=req, positions=positions)
        if not at:
            assert torch.all(out[t] == 0) and torch.all(torch.isneginf(lse[t]))
            continue
        kv, qd = vals[at], q[t].double()
        x = qd @ kv.T * SCALE
        rlse = torch.logsumexp(x, 1)
        w = torch.exp(x - rlse[:, None])
        ref = w @ kv
        # tolerance() with the mean of |kv_j - ref| bounded by its root mean square, and 2^-12 of w |kv| for the
        # sums of 16384 rows (half of 1024 steps of at most 2^-21)
        ex = 64 * 2.0 ** -23 * SCALE * (qd.abs() @ kv.abs().T).amax(1) + 2.0 ** -20
        spread = (w @ kv ** 2 - ref ** 2).clamp_min(0).sqrt()
        eta = 2 * (2.0 ** -11 + 2 * ex)
        half = torch.finfo(DT[dtype]).eps / 2
        tol = (eta[:, None] * spread + 2.0 ** -12 * (w @ kv.abs()) + len(at) * 2.0 ** -29 * kv.abs().max() +
               half * 1.01 * ref.abs() + 2.0 ** -25)
        worst = ((out[t].double() - ref).abs() / tol).max().item()
        assert worst <= 1, (t, len(at), worst)
        assert torch.all((lse[t].double() - rlse).abs() <= 2 * ex + 2.0 ** -13 + 2.0 ** -20 * (1 + x.abs().amax(1)))


@pytest.mark.parametrize("T,max_rows", [(1, 1), (5, 64), (152, 33), (3000, 64)])
def test_attn_workspace_of_tokens_that_are_never_split(T, max_rows):
    """Up to 64 rows a token is one chunk, which no second block works on: no room for parts is asked for."""
    rng = np.random.default_rng(62)
    need = ds4x.kv4_attn_workspace_bytes(T, max_rows)
    assert need <= 65536
    assert ds4x.kv4_attn_workspace_bytes(T, 65) > need
    pool = Pool(rng, [max_rows], 1)
    q = queries(rng, min(T, 8), "f16").repeat((T + 7) // 8, 1, 1)[:T].contiguous()
    buf = torch.full((need + 4096,), 173, dtype=torch.uint8, device="cuda")
    lists = dict(req=np.zeros(T, np.int32))
    out, lse = ds4x.kv4_attn(q, *pool.dev, 1, req=i32(lists["req"]), workspace=buf[:need])
    assert torch.all(buf[need:] == 173)
    some = np.unique([0, T // 2, T - 1])
    check_attn(q[some], pool, out[some], lse[some], SCALE, "f16", dict(req=lists["req"][some]))


@pytest.mark.parametrize("T,dtype", [(7, "bf16"), (9, "f16"), (37, "f16"), (38, "bf16"), (64, "f16")])
def test_attn_one_long_request_among_short_ones(T, dtype):
    """Its parts lie in most of the blocks, whichever form of the joining kernel the number of tokens picks."""
    rng = np.random.default_rng(T)
    rows = rng.integers(0, 65, T)
    rows[T // 2] = 9000 + T
    pool = Pool(rng, rows, 32)
    q = queries(rng, T, dtype)
    out, lse = run_attn(q, pool)
    some = np.array([0, T // 2 - 1, T // 2, T // 2 + 1, T - 1])
    check_attn(q[some], pool, out[some], lse[some], SCALE, dtype, dict(req=some.astype(np.int32)))
    o2, l2 = run_attn(q, pool)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
