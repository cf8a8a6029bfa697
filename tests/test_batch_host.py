"""The batch operators on a host without a GPU: their refusals come before any CUDA call,
vg_rope_freqs agrees with the formula, and the oracle's own pool and rotation are pinned to
facts that do not come from them."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

import oracle
from self_speculative_sparse_gb300 import binding as vb
from self_speculative_sparse_gb300 import build
from tests.test_abi import A, MIS, Buf, cache, dims


@pytest.fixture(scope="module")
def lib():
    build.build()
    return vb.load()


# ------------------------------------------------------------ rotary positions
def rope_call(lib, d=None, c=None, rot=64, layout=0, mscale=1.0, freq=A, q=A, k=A, v=A, q_stride=512, k_stride=128,
              v_stride=128, row_start=A, n_rows=4, prefix_len=A, q_out=A, q_out_stride=512, status=None, rope=True):
    d = dims() if d is None else d
    c = cache() if c is None else c
    r = vb.vg_rope(vb.ptr(freq), rot, layout, mscale)
    return lib.vg_rope_append(ctypes.byref(d), ctypes.byref(c), ctypes.byref(r) if rope else None, vb.ptr(q), q_stride,
                              vb.ptr(k), k_stride, vb.ptr(v), v_stride, vb.ptr(row_start), n_rows, vb.ptr(prefix_len),
                              vb.ptr(q_out), q_out_stride, vb.ptr(status), None)


@pytest.mark.parametrize("bad", [
    dict(rope=False), dict(freq=None), dict(freq=MIS), dict(rot=0), dict(rot=3), dict(rot=66), dict(layout=2),
    dict(mscale=float("nan")), dict(q=None), dict(k=None), dict(v=None), dict(q_out=None), dict(prefix_len=None),
    dict(q=MIS), dict(k=MIS), dict(v=MIS), dict(q_out=MIS), dict(row_start=MIS), dict(prefix_len=MIS),
    dict(q_stride=511), dict(q_stride=504), dict(k_stride=120), dict(v_stride=64), dict(q_out_stride=520, q_out=A),
    dict(n_rows=-1), dict(n_rows=(1 << 24) + 1), dict(row_start=None, n_rows=5), dict(status=Buf(0x10002)),
    dict(d=dims(scale=-1.0)),
])
def test_rope_refusals(lib, bad):
    assert rope_call(lib, **bad) == vb.VG_ERR_INVALID_ARG
    assert lib.vg_last_error()


def test_rope_unsupported_shapes(lib):
    assert rope_call(lib, d=dims(d=80)) == vb.VG_ERR_UNSUPPORTED_SHAPE
    assert rope_call(lib, d=dims(B=0)) == vb.VG_ERR_UNSUPPORTED_SHAPE


def test_rope_of_no_rows_is_nothing(lib):
    assert rope_call(lib, n_rows=0) == vb.VG_OK


@pytest.mark.parametrize("scaling", ["plain", "linear", "base", "ramp"])
@pytest.mark.parametrize("rot,base,factor", [(2, 10000.0, 4.0), (6, 10000.0, 2.0), (64, 500000.0, 8.0),
                                             (128, 1e6, 32.0)])
def test_rope_freqs_are_the_formula_in_turns(lib, scaling, rot, base, factor):
    kind = dict(plain=vb.VG_ROPE_PLAIN, linear=vb.VG_ROPE_LINEAR, base=vb.VG_ROPE_BASE, ramp=vb.VG_ROPE_RAMP)[scaling]
    got = vb.vg_rope_freqs(rot, base, kind, factor, 8192.0, 1.0, 32.0)
    want = oracle.rope_inverse(rot, base, scaling, factor, 8192.0) / (2 * math.pi)
    # both sides are a few float64 operations: 2^-48 relative covers pow, two products and the
    # division; the fixed-point rounding is half a step of 2^-64
    for g, w in zip(got.tolist(), want.tolist()):
        assert abs(Fraction(g, 1 << 64) - Fraction(w)) <= Fraction(w) * Fraction(1, 1 << 48) + Fraction(1, 1 << 65)


@pytest.mark.parametrize("bad", [
    dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=2000), dict(base=0.0), dict(base=float("inf")), dict(scaling=4),
    dict(scaling=1, factor=0.0), dict(scaling=2, factor=float("nan")), dict(scaling=3, factor=2.0, orig_len=0.0),
    dict(scaling=3, factor=2.0, orig_len=10.0, slow=4.0, fast=4.0), dict(base=1e-9), dict(scaling=1, factor=0.1),
])
def test_rope_freqs_refusals(lib, bad):
    kw = dict(rot_dim=64, base=10000.0)
    kw.update(bad)
    with pytest.raises(vb.VgError) as e:
        vb.vg_rope_freqs(**kw)
    assert e.value.status == vb.VG_ERR_INVALID_ARG


def test_oracle_rope_keeps_norms_and_depends_on_the_distance_only():
    r = np.random.default_rng(4)
    inv = oracle.rope_inverse(16, 10000.0)
    x, y = r.standard_normal((1, 2, 24)), r.standard_normal((1, 2, 24))
    for inter in (False, True):
        a = oracle.rope(x, np.array([70]), inv, inter)
        assert np.allclose(np.linalg.norm(a, axis=-1), np.linalg.norm(x, axis=-1))
        assert np.array_equal(a[..., 16:], x[..., 16:])
        d1 = (oracle.rope(x, np.array([12]), inv, inter) * oracle.rope(y, np.array([5]), inv, inter)).sum()
        d2 = (oracle.rope(x, np.array([1007]), inv, inter) * oracle.rope(y, np.array([1000]), inv, inter)).sum()
        assert abs(d1 - d2) < 1e-9
    assert np.allclose(oracle.rope(x, np.array([0]), inv, False), x)


# ------------------------------------------------------------ page pool
def pool(**kw):
    base = dict(page_table=A.addr, held=A.addr, refs=A.addr, n_seqs=8, pages_per_seq=16, n_pages=64, page_size=16)
    base.update(kw)
    return vb.vg_page_pool(**base)


@pytest.mark.parametrize("bad", [
    dict(page_table=None), dict(held=None), dict(refs=None), dict(page_table=MIS.addr), dict(refs=MIS.addr),
    dict(n_seqs=0), dict(n_seqs=65537), dict(pages_per_seq=0), dict(pages_per_seq=1 << 28), dict(n_pages=0),
    dict(page_size=0), dict(page_size=(1 << 20) + 1), dict(n_pages=1 << 27, page_size=16),
])
def test_pool_refusals(lib, bad):
    p = pool(**bad)
    assert lib.vg_pages_workspace_size(ctypes.byref(p)) == 0
    assert lib.vg_pages_resize(ctypes.byref(p), A.addr, A.addr, 1, A.addr, 1 << 30, None, None) == vb.VG_ERR_INVALID_ARG


def test_pool_workspace_is_checked(lib):
    p = pool()
    need = lib.vg_pages_workspace_size(ctypes.byref(p))
    assert need > 0

    def call(ws, size):
        return lib.vg_pages_resize(ctypes.byref(p), A.addr, A.addr, 1, ws, size, None, None)
    assert call(None, need) == vb.VG_ERR_WORKSPACE
    assert call(0x10010, need) == vb.VG_ERR_WORKSPACE
    assert call(0x10000, need - 1) == vb.VG_ERR_WORKSPACE


def test_resize_refusals(lib):
    p = pool()

    def call(seq=A, length=A, n=2, status=None):
        return lib.vg_pages_resize(ctypes.byref(p), vb.ptr(seq), vb.ptr(length), n, 0x10000, 1 << 30, vb.ptr(status), None)
    assert call(n=0) == vb.VG_OK
    for bad in (dict(n=-1), dict(n=9), dict(length=None), dict(length=MIS), dict(seq=MIS), dict(status=Buf(0x10002))):
        assert call(**bad) == vb.VG_ERR_INVALID_ARG, bad
    assert lib.vg_pages_resize(None, A.addr, A.addr, 1, A.addr, 1 << 30, None, None) == vb.VG_ERR_INVALID_ARG


def test_fork_and_compact_refusals(lib):
    p = pool()
    good = (vb.vg_kv_cache * 1)(vb.vg_kv_cache(A.addr, A.addr, None, 64 * 16, None, 0, 0))
    small = (vb.vg_kv_cache * 1)(vb.vg_kv_cache(A.addr, A.addr, None, 64 * 16 - 1, None, 0, 0))
    null = (vb.vg_kv_cache * 1)(vb.vg_kv_cache(A.addr, None, None, 64 * 16, None, 0, 0))
    skew = (vb.vg_kv_cache * 1)(vb.vg_kv_cache(MIS.addr, A.addr, None, 64 * 16, None, 0, 0))

    def fork(caches=good, layers=1, token=2048, parent=A, child=A, length=A, n=2, room=1):
        return lib.vg_pages_fork(ctypes.byref(p), caches, layers, token, vb.ptr(parent), vb.ptr(child), vb.ptr(length),
                                 n, room, 0x10000, 1 << 30, None, None)

    def compact(caches=good, layers=1, token=2048, table=A, refs=A, live=A):
        return lib.vg_pages_compact(ctypes.byref(p), caches, layers, token, vb.ptr(table), vb.ptr(refs), vb.ptr(live),
                                    0x10000, 1 << 30, None, None)
    assert fork(n=0) == vb.VG_OK
    for bad in (dict(caches=small), dict(caches=null), dict(caches=skew), dict(caches=None), dict(token=8),
                dict(token=24), dict(token=(1 << 20) + 16)):
        assert fork(**bad) == vb.VG_ERR_INVALID_ARG, bad
        assert compact(**bad) == vb.VG_ERR_INVALID_ARG, bad
    for layers in (0, 129):
        assert fork(layers=layers) == vb.VG_ERR_UNSUPPORTED_SHAPE
        assert compact(layers=layers) == vb.VG_ERR_UNSUPPORTED_SHAPE
    for bad in (dict(parent=None), dict(child=None), dict(length=None), dict(parent=MIS), dict(n=9), dict(n=-1),
                dict(room=-1)):
        assert fork(**bad) == vb.VG_ERR_INVALID_ARG, bad
    for bad in (dict(table=None), dict(refs=None), dict(live=None), dict(table=MIS), dict(table=Buf(A.addr + 16)),
                dict(refs=Buf(A.addr + 16))):
        assert compact(**bad) == vb.VG_ERR_INVALID_ARG, bad


def test_oracle_pool_shares_copies_and_runs_out():
    p = oracle.Pool(4, 4, 6, 8)
    p.resize([0], [20])
    assert p.rows[0] == [0, 1, 2] and p.refs == [1, 1, 1, 0, 0, 0]
    assert p.fork([0, 0], [1, 2], [20, 16], 0) == [(2, 3, 4)]
    assert p.rows[1] == [0, 1, 3] and p.rows[2] == [0, 1] and p.refs == [3, 3, 1, 1, 0, 0]
    p.resize([3], [25])
    assert p.errors == ["pages"] and p.rows[3] == []
    p.resize([0, 3], [0, 17])
    assert p.rows[3] == [2, 4, 5] and p.refs == [2, 2, 1, 1, 1, 1]
    p.resize([1, 2], [0, 0])
    assert p.compact() == [(4, 0), (5, 1)] and p.rows[3] == [2, 0, 1]


# ------------------------------------------------------------ shared prefixes
def shared_call(lib, d=None, c=None, ng=2, start=A, shared=A, groups=True, q=A, kn=A, vn=A, prefix=A, mask=0x9, scores=A,
                stride=512, out=A, ws=A, ws_bytes=1 << 40, status=None):
    d = dims() if d is None else d
    c = cache() if c is None else c
    g = vb.vg_prefix_groups(ng, vb.ptr(start), vb.ptr(shared))
    return lib.vg_shared_verify_attn(ctypes.byref(d), ctypes.byref(c), ctypes.byref(g) if groups else None, vb.ptr(q),
                                     vb.ptr(kn), vb.ptr(vn), vb.ptr(prefix), mask, vb.ptr(scores), stride, vb.ptr(out),
                                     vb.ptr(ws), ws_bytes, vb.ptr(status), None)


@pytest.mark.parametrize("bad", [
    dict(groups=False), dict(ng=0), dict(ng=1025), dict(start=None), dict(shared=None), dict(start=MIS), dict(shared=MIS),
    dict(q=None), dict(prefix=None), dict(out=None), dict(kn=None), dict(vn=None), dict(q=MIS), dict(out=MIS),
    dict(mask=0x10), dict(mask=0), dict(scores=None), dict(stride=511), dict(scores=MIS), dict(status=Buf(0x10002)),
    dict(d=dims(max_len=-1)),
])
def test_shared_refusals(lib, bad):
    assert shared_call(lib, **bad) == vb.VG_ERR_INVALID_ARG
    assert lib.vg_last_error()


def test_shared_unsupported_shapes_and_no_gpu(lib):
    import torch
    assert shared_call(lib, d=dims(d=80)) == vb.VG_ERR_UNSUPPORTED_SHAPE
    assert shared_call(lib, d=dims(gamma=16)) == vb.VG_ERR_UNSUPPORTED_SHAPE
    odd = vb.vg_kv_cache(A.addr, A.addr, None, 4096, A.addr, 24, 30)
    assert shared_call(lib, c=odd) == vb.VG_ERR_UNSUPPORTED_SHAPE
    if not torch.cuda.is_available():
        assert shared_call(lib) == vb.VG_ERR_CUDA
        assert shared_call(lib, ng=1, start=None) == vb.VG_ERR_CUDA
        g = vb.vg_prefix_groups(1, None, A.addr)
        assert lib.vg_shared_verify_workspace_size(ctypes.byref(dims()), ctypes.byref(g)) == 0
