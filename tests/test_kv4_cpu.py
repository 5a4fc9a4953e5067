"""The paged 4-bit cache without a GPU: pins of the plain implementation, and refusals."""
import ctypes

import numpy as np
import pytest
import torch

import deepseek_v4_sparse_gb300 as ds4x
from deepseek_v4_sparse_gb300 import build as ds4x_build
from oracle import kv4

A = 0x10000  # an aligned, never dereferenced address: validation fails before any use


@pytest.fixture(scope="module")
def lib():
    ds4x_build.build()
    return ds4x.load()


def _p(v):
    return ctypes.c_void_p(v)


# ------------------------------------------------------------------------------ the oracle itself
def test_quantise_known_group():
    x = np.zeros((1, 512))
    # top 6 -> e = 0: every grid value is kept, ties go to the even code
    x[0, :12] = [6, -4, 3, 2, 1.5, 1, 0.5, 0.25, 0.75, 2.5, 3.5, -5]
    x[0, 32] = 6.25     # over 6 * 2^0: e = 1, 3.125 -> 3
    x[0, 64] = 1e9      # saturates
    x[0, 96] = 1e-12    # below half of the least value
    codes, scales = kv4.quantise(x)
    v = kv4.values(codes, scales)
    assert v[0, :12].tolist() == [6, -4, 3, 2, 1.5, 1, 0.5, 0, 1, 2, 4, -4]
    assert scales[0, :4].tolist() == [127, 128, 140, 104]
    assert v[0, 32] == 6 and v[0, 64] == 49152 and v[0, 96] == 0
    assert np.all(scales[0, 4:] == 104)


def test_values_survive_a_second_quantisation():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 512)) * np.exp2(rng.integers(-20, 12, (5, 1)).astype(float))
    once = kv4.values(*kv4.quantise(x))
    assert np.array_equal(kv4.values(*kv4.quantise(once)), once)
    # the grid's widest gap is 2 (4 to 6) at a top of at least 3: within a sixth of the group's top
    top = np.abs(x).reshape(5, 16, 32).max(-1).repeat(32, 1)
    assert np.all(np.abs(once - x) <= top / 3 + 2.0 ** -24)


def test_values_are_exact_in_both_16_bit_types():
    codes = np.tile(np.arange(256, dtype=np.uint8), (37, 1))
    scales = np.repeat(np.arange(104, 141, dtype=np.uint8)[:, None], 16, 1)
    v = torch.from_numpy(kv4.values(codes, scales))
    for dt in (torch.float16, torch.bfloat16):
        assert torch.equal(v.to(dt).double(), v)


def test_page_plan_by_hand():
    tables = np.array([[5, -1, -1], [-1, -1, -1]], dtype=np.int32)
    out = kv4.page_plan([6, 0], [9, 5], [3, 0], tables, [9, 8, 7], 3, 2, 4, 16, 10)
    positions, req, slots, tab, seen, rows, left, totals = out
    assert positions[:14].tolist() == list(range(6, 15)) + list(range(5)) and (positions[14:] == -1).all()
    assert req.tolist() == [0] * 9 + [1] * 5 + [-1] * 2
    # request 0: rows 3..6 (page 5 is filled up, then page 7); request 1: rows 0, 1 on page 8
    assert slots.tolist() == [23, 28, 29, 30, 32, 33, -1, -1, -1, -1]
    assert tab.tolist() == [[5, 7, -1], [8, -1, -1]]
    assert seen.tolist() == [15, 5] and rows.tolist() == [7, 2] and left == 1
    assert totals.tolist() == [14, 6, 6, 2]


def test_attention_of_one_row_is_the_row():
    rng = np.random.default_rng(2)
    pool = rng.standard_normal((8, 512))
    tables = np.array([[1]], dtype=np.int32)
    out, lse = kv4.attn(rng.standard_normal((1, 64, 512)), pool, 0.1, tables=tables, rows=[2], page_rows=4,
                        indices=np.array([[1, -1, 2]]))
    assert np.array_equal(out[0], np.tile(pool[5], (64, 1)))  # row 2 is not held
    assert np.isfinite(lse).all()


# ------------------------------------------------------------------------------------- refusals
def _plan(lib, n_req=4, max_pages=8, page_rows=16, ratio=4, T_cap=10, R_cap=10, free_cap=5, seen=A, tables=A, nf=A,
          positions=A, slots=A):
    return lib.ds4x_page_plan(_p(seen), _p(A), _p(A), _p(tables), _p(A), free_cap, _p(nf), n_req, max_pages, page_rows,
                              ratio, T_cap, R_cap, _p(positions), _p(A), _p(slots), None, None, None, None, None)


def test_page_plan_refusals(lib):
    for bad in (dict(n_req=-1), dict(max_pages=-1), dict(page_rows=0), dict(ratio=0), dict(T_cap=-1), dict(R_cap=-1),
                dict(free_cap=-1), dict(seen=None), dict(tables=None), dict(nf=None), dict(positions=None),
                dict(slots=None), dict(seen=A + 2), dict(n_req=0)):
        assert _plan(lib, **bad) == ds4x.ERR_INVALID, bad
    for bad in (dict(n_req=ds4x.MAX_REQ + 1), dict(page_rows=24), dict(page_rows=2 * ds4x.MAX_PAGE_ROWS),
                dict(max_pages=1 << 28, page_rows=16)):
        assert _plan(lib, **bad) == ds4x.ERR_UNSUPPORTED, bad
    assert _plan(lib, n_req=0, T_cap=0, R_cap=0) == ds4x.OK


def test_append_and_read_refusals(lib):
    def append(rows=A, dtype=0, slots=A, n=3, D=512, codes=A, scales=A, n_slots=9):
        return lib.ds4x_kv4_append(_p(rows), dtype, _p(slots), n, D, _p(codes), _p(scales), n_slots, None)

    def read(rows=A, dtype=0, slots=A, n=3, D=512, codes=A, scales=A, n_slots=9):
        return lib.ds4x_kv4_read(_p(codes), _p(scales), n_slots, _p(slots), n, D, _p(rows), dtype, None)

    for f in (append, read):
        for bad in (dict(n=-1), dict(D=0), dict(n_slots=-1), dict(dtype=2), dict(rows=None), dict(slots=None),
                    dict(codes=None), dict(scales=None), dict(rows=A + 8), dict(codes=A + 4), dict(scales=A + 8),
                    dict(slots=A + 1)):
            assert f(**bad) == ds4x.ERR_INVALID, bad
        assert f(D=128) == ds4x.ERR_UNSUPPORTED
        assert f(n=0, rows=None) == ds4x.OK


def _attn(lib, q=A, dtype=1, codes=A, scales=A, n_slots=64, tables=A, rows=A, n_req=2, max_pages=4, page_rows=16,
          req=A, positions=A, ratio=4, indices=A, counts=None, T=4, Hq=64, D=512, k_top=512, out=A, lse=None, ws=A,
          nbytes=1 << 40):
    return lib.ds4x_kv4_attn(_p(q), dtype, _p(codes), _p(scales), n_slots, _p(tables), _p(rows), n_req, max_pages,
                             page_rows, _p(req), _p(positions), ratio, _p(indices), _p(counts), T, Hq, D, k_top, 0.1,
                             _p(out), _p(lse), _p(ws), nbytes, None)


def test_attn_refusals(lib):
    for bad in (dict(T=-1), dict(Hq=0), dict(D=-2), dict(n_slots=-1), dict(n_req=-1), dict(max_pages=-1),
                dict(page_rows=0), dict(ratio=0), dict(k_top=0), dict(dtype=9), dict(q=None), dict(out=None),
                dict(q=A + 2), dict(out=A + 8), dict(lse=A + 4), dict(codes=None), dict(scales=A + 1),
                dict(tables=None), dict(rows=None), dict(req=A + 2), dict(indices=A + 1), dict(req=None, n_req=3)):
        assert _attn(lib, **bad) == ds4x.ERR_INVALID, bad
    for bad in (dict(Hq=32), dict(D=256), dict(page_rows=48), dict(k_top=ds4x.MAX_KTOP + 1),
                dict(max_pages=1 << 28, page_rows=16)):
        assert _attn(lib, **bad) == ds4x.ERR_UNSUPPORTED, bad
    assert _attn(lib, T=0, q=None) == ds4x.OK
    assert ds4x.kv4_attn_workspace_bytes(0, 512) == 0 and ds4x.kv4_attn_workspace_bytes(5, 0) == 0
    if ds4x.kv4_attn_workspace_bytes(4, 512):
        assert _attn(lib, nbytes=16) == ds4x.ERR_WORKSPACE
        assert _attn(lib, ws=None) == ds4x.ERR_WORKSPACE
        assert _attn(lib, ws=A + 8) == ds4x.ERR_INVALID


def test_binding_refuses_host_tensors():
    z = torch.zeros(4, dtype=torch.int32)
    pool = torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((4, 16), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        ds4x.kv4_append(torch.zeros((4, 512), dtype=torch.float16), z, *pool)
    with pytest.raises(ValueError, match="CUDA"):
        ds4x.kv4_read(*pool, z, torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        ds4x.page_plan(z, z, z, z.reshape(4, 1), z, z, 4, 16, 4, 4)
    with pytest.raises(ValueError, match="CUDA"):
        ds4x.kv4_attn(torch.zeros((1, 64, 512), dtype=torch.float16), *pool, z.reshape(4, 1), z, 16)
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        ds4x.kv4_append(torch.zeros((4, 512)), z, *pool)


def test_page_plan_by_hand_after_a_shortage():
    """Ratio 4, ten rows held; no page for the rows behind the second page's end, pages again in the next step."""
    tables = np.array([[0, 1, 2, -1, -1, -1, -1, -1]], dtype=np.int32)
    out = kv4.page_plan([40], [40], [10], tables, [9, 8], 0, 4, 4, 40, 12)
    slots, tab, seen, rows, left, totals = out[2:]
    assert slots.tolist() == [10, 11] + [-1] * 10 and seen.tolist() == [80] and rows.tolist() == [12]
    assert totals.tolist() == [40, 10, 2, 0]
    # pooled rows 20..29 may not become rows 12..21: none gets a slot, no page is taken, what is held stays
    out = kv4.page_plan(seen, [40], rows, tab, [9, 8, 7], 3, 4, 4, 40, 12)
    slots, tab2, seen, rows, left, totals = out[2:]
    assert slots.tolist() == [-1] * 12 and seen.tolist() == [120] and rows.tolist() == [12] and left == 3
    assert np.array_equal(tab, tab2) and totals.tolist() == [40, 10, 0, 0]
    # taken back to its last row, it goes on
    out = kv4.page_plan([48], [8], rows, tab2, [9, 8, 7], 3, 4, 4, 8, 4)
    assert out[2].tolist() == [28, 29, -1, -1] and out[5].tolist() == [14] and out[6] == 2


def test_wait_sites_name_one_kernel():
    """The status word tells which wait gave up: no two source files share a number."""
    import os
    import re
    csrc = os.path.join(os.path.dirname(ds4x_build.__file__), "csrc")
    of = {}
    for name in sorted(os.listdir(csrc)):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(csrc, name)).read())
        for site in re.findall(r"status, (0x[0-9a-f]+|\d+)(?:, timeout_ns)?\)", text):
            of.setdefault(int(site, 0), set()).add(name)
    assert len(of) > 30
    shared = {site: files for site, files in of.items() if len(files) > 1}
    assert not shared, shared
