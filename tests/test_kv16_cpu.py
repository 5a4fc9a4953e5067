"""The paged 16-bit cache without a GPU: pins of the plain implementation, and refusals."""
import ctypes

import numpy as np
import pytest
import torch

import deepseek_v4_sparse_gb300 as ds4x
from deepseek_v4_sparse_gb300 import build as ds4x_build
from oracle import kv16

A = 0x10000  # an aligned, never dereferenced address: validation fails before any use


@pytest.fixture(scope="module")
def lib():
    ds4x_build.build()
    return ds4x.load()


def _p(v):
    return ctypes.c_void_p(v)


# ------------------------------------------------------------------------------ the oracle itself
def test_rotate_by_a_quarter_turn():
    x = np.arange(1.0, 9.0)[None, :]
    y = kv16.rotate(x, [3], [np.pi / 6, np.pi / 3])         # 90 and 180 degrees, the first four stay
    assert np.allclose(y, [[1, 2, 3, 4, -6, 5, -7, -8]], atol=1e-14)
    assert np.allclose(kv16.rotate(y, [3], [np.pi / 6, np.pi / 3], inverse=True), x, atol=1e-14)


def test_rotated_products_depend_on_the_distance_alone():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 16))
    f = 10.0 ** -np.arange(8)
    dot = lambda a, b: float(kv16.rotate(q, [a], f)[0] @ kv16.rotate(k, [b], f)[0])  # noqa: E731
    assert np.isclose(dot(7, 3), dot(1007, 1003)) and not np.isclose(dot(7, 3), dot(7, 4))


def test_rows_seen_by_hand():
    tables = np.array([[2, 0, -1, 1]], dtype=np.int32)
    see = lambda **kw: kv16.seen_rows(0, tables, [13], 4, 12, req=[0], **kw)  # noqa: E731
    assert see()[1] == [0, 1, 2, 3, 4, 5, 6, 7, 12] and see()[2] == [8, 9, 10, 11, 0, 1, 2, 3, 4]
    assert see(positions=[5])[1] == [0, 1, 2, 3, 4, 5] and see(positions=[5])[0] == 6
    assert see(positions=[5], window=2)[1] == [4, 5]
    assert see(positions=[5], window=4, first=[3])[1] == [3, 4, 5]
    assert see(positions=[1], prefix=[5])[1] == [0, 1, 2, 3, 4]
    assert see(positions=[1], prefix=[5], window=1)[1] == [1, 2, 3, 4]
    assert see(positions=[23], ratio=4)[1] == [0, 1, 2, 3, 4, 5]
    assert see(positions=[-1], prefix=[5])[1] == [] and see(positions=[40], window=3)[1] == []


def test_attention_sink_and_join_by_hand():
    pool = np.zeros((4, 8))
    pool[1, 0], pool[2, 0] = 1.0, 3.0
    tables, q = np.array([[0]], dtype=np.int32), np.zeros((1, 2, 8))
    lists = dict(tables=tables, rows=[4], page_rows=4, first=[1], positions=[2])
    out, lse = kv16.attn(q, pool, 1.0, **lists)
    assert np.allclose(out[0, :, 0], 2.0) and np.allclose(lse, np.log(2))
    out, lse = kv16.attn(q, pool, 1.0, sinks=[np.log(2.0), -np.inf], **lists)
    assert np.allclose(out[0, :, 0], [1.0, 2.0]) and np.allclose(lse, [np.log(4), np.log(2)])
    other = np.full((1, 2, 8), 5.0), np.array([[np.log(2.0), -np.inf]])
    out, lse = kv16.attn(q, pool, 1.0, other=other, **lists)
    assert np.allclose(out[0, :, 0], [3.5, 2.0]) and np.allclose(lse, [np.log(4), np.log(2)])
    out, lse = kv16.attn(q, pool, 1.0, slopes=[np.log(3.0), 0.0], **lists)
    assert np.allclose(out[0, :, 0], [(1 / 3 + 3) / (4 / 3), 2.0])


# ------------------------------------------------------------------------------------- refusals
def test_rotate_refusals(lib):
    def rotate(x=A, dtype=0, pos=A, f=A, T=3, H=2, D=64, rot=8, out=A):
        return lib.ds4x_rotate(_p(x), dtype, _p(pos), _p(f), T, H, D, rot, 0, _p(out), None)

    for bad in (dict(T=-1), dict(H=-1), dict(D=0), dict(rot=0), dict(rot=7), dict(rot=66), dict(dtype=2), dict(x=None),
                dict(out=None), dict(pos=None), dict(f=None), dict(x=A + 8), dict(out=A + 4), dict(pos=A + 2),
                dict(f=A + 4)):
        assert rotate(**bad) == ds4x.ERR_INVALID, bad
    for bad in (dict(D=66), dict(D=8192, rot=ds4x.MAX_ROT + 2), dict(H=1 << 26)):
        assert rotate(**bad) == ds4x.ERR_UNSUPPORTED, bad
    assert rotate(T=0, x=None) == ds4x.OK and rotate(H=0, x=None) == ds4x.OK


def test_append_refusals(lib):
    def append(rows=A, dtype=0, slots=A, pos=A, f=A, n=3, D=512, rot=64, pool=A, n_slots=9):
        return lib.ds4x_kv16_append(_p(rows), dtype, _p(slots), _p(pos), _p(f), n, D, rot, _p(pool), n_slots, None)

    for bad in (dict(n=-1), dict(D=0), dict(n_slots=-1), dict(dtype=2), dict(rot=-2), dict(rot=63), dict(rot=514),
                dict(rows=None), dict(slots=None), dict(pool=None), dict(pos=None), dict(f=None), dict(rows=A + 8),
                dict(pool=A + 4), dict(slots=A + 1), dict(pos=A + 2), dict(f=A + 4)):
        assert append(**bad) == ds4x.ERR_INVALID, bad
    assert append(D=128) == ds4x.ERR_UNSUPPORTED
    assert append(n=0, rows=None) == ds4x.OK


def _attn(lib, q=A, dtype=1, pool=A, n_slots=64, tables=A, rows=A, n_req=2, max_pages=4, page_rows=16, req=A,
          positions=A, ratio=1, window=0, first=None, prefix=None, T=4, Hq=64, D=512, cap=0.0, slopes=None, sinks=None,
          oo=None, ol=None, out=A, lse=None, ws=A, nbytes=1 << 40):
    return lib.ds4x_kv16_attn(_p(q), dtype, _p(pool), n_slots, _p(tables), _p(rows), n_req, max_pages, page_rows,
                              _p(req), _p(positions), ratio, window, _p(first), _p(prefix), T, Hq, D, 0.1, cap,
                              _p(slopes), _p(sinks), _p(oo), _p(ol), _p(out), _p(lse), _p(ws), nbytes, None)


def test_attn_refusals(lib):
    for bad in (dict(T=-1), dict(Hq=0), dict(D=-2), dict(n_slots=-1), dict(n_req=-1), dict(max_pages=-1),
                dict(page_rows=0), dict(ratio=0), dict(window=-1), dict(cap=-1.0), dict(cap=float("nan")),
                dict(cap=float("inf")), dict(dtype=9), dict(q=None), dict(out=None), dict(q=A + 2), dict(out=A + 8),
                dict(lse=A + 4), dict(pool=None), dict(pool=A + 8), dict(tables=None), dict(rows=None),
                dict(req=A + 2), dict(positions=A + 1), dict(first=A + 2), dict(prefix=A + 3), dict(slopes=A + 1),
                dict(sinks=A + 2), dict(oo=A), dict(ol=A), dict(oo=A + 8, ol=A), dict(oo=A, ol=A + 2),
                dict(req=None, n_req=3)):
        assert _attn(lib, **bad) == ds4x.ERR_INVALID, bad
    for bad in (dict(Hq=32), dict(D=256), dict(page_rows=48), dict(page_rows=2 * ds4x.MAX_PAGE_ROWS),
                dict(max_pages=1 << 28, page_rows=16)):
        assert _attn(lib, **bad) == ds4x.ERR_UNSUPPORTED, bad
    assert _attn(lib, T=0, q=None) == ds4x.OK
    assert ds4x.kv16_attn_workspace_bytes(0, 512) == 0 and ds4x.kv16_attn_workspace_bytes(5, 0) == 0
    assert ds4x.kv16_attn_workspace_bytes(4, 64) == 0 and ds4x.kv16_attn_workspace_bytes(4, 1024) > 16
    for bad in (dict(nbytes=16), dict(ws=None)):
        assert _attn(lib, max_pages=64, page_rows=16, **bad) == ds4x.ERR_WORKSPACE, bad
    assert _attn(lib, max_pages=64, page_rows=16, ws=A + 8) == ds4x.ERR_INVALID


def test_attn_refuses_scales_that_leave_fp32(lib):
    def attn(scale):  # pages of 48 rows: what is let through is refused for them
        return lib.ds4x_kv16_attn(_p(A), 1, _p(A), 64, _p(A), _p(A), 2, 4, 48, _p(A), _p(A), 1, 0, None, None, 4, 64, 512,
                                  scale, 0.0, None, None, None, None, _p(A), None, None, 0, None)

    for bad in (float("nan"), float("inf"), -float("inf"), 1.8e38, -3.4e38):
        assert attn(bad) == ds4x.ERR_INVALID, bad
    for ok in (0.0, -1.0, 2.0 ** 127, -2.0 ** 127):
        assert attn(ok) == ds4x.ERR_UNSUPPORTED, ok


def test_binding_refuses_host_tensors():
    z = torch.zeros(4, dtype=torch.int32)
    f = torch.zeros(2, dtype=torch.float64)
    x = torch.zeros((4, 512), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        ds4x.rotate(x, z, f)
    with pytest.raises(ValueError, match="CUDA"):
        ds4x.kv16_append(x, z, x.clone())
    with pytest.raises(ValueError, match="CUDA"):
        ds4x.kv16_attn(torch.zeros((1, 64, 512), dtype=torch.float16), x, z.reshape(4, 1), z, 16)
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        ds4x.rotate(x.float(), z, f)
