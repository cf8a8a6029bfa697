"""Requests to the batch operators as the Python classes take them, on a host without a GPU: empty ones do
nothing, and tensors that do not fit are refused before any call."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from self_speculative_sparse_gb300 import binding as vb  # noqa: E402
from self_speculative_sparse_gb300 import build  # noqa: E402
from tests.test_abi import A, cache, dims  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def make_pool(layers=2, n_seqs=6, n_pages=12, page=4, **kw):
    from self_speculative_sparse_gb300.runtime import PagePool
    kv = [tuple(torch.zeros(n_pages * page, 2, 64, dtype=torch.bfloat16) for _ in range(2)) for _ in range(layers)]
    pool = PagePool(n_seqs, 5, n_pages, page, kw.get("kv", kv))
    ws = torch.empty(pool.ws.numel() + 256, dtype=torch.uint8)  # (host memory is not always 256-byte aligned)
    pool.ws = ws[-ws.data_ptr() % 256:][:pool.ws.numel()]
    return pool


def empty():
    return torch.empty(0, dtype=torch.int32)


def test_empty_requests_do_nothing():
    pool = make_pool()
    assert empty().data_ptr() == 0
    pool.resize(empty(), empty(), stream=0)
    pool.resize(None, empty(), stream=0)
    pool.fork(empty(), empty(), empty(), 3, stream=0)


def test_no_rows_rotate_to_nothing():
    d, c, r = dims(), cache(), vb.vg_rope(A.addr, 64, 0, 1.0)
    rows = torch.empty(0, 8, 64, dtype=torch.bfloat16)
    keys = torch.empty(0, 2, 64, dtype=torch.bfloat16)
    vb.vg_rope_append(d, c, r, rows, rows.stride(0), keys, keys.stride(0), keys, keys.stride(0), A, 0, A, rows,
                      rows.stride(0), stream=0)
    st = vb.load().vg_rope_append(ctypes.byref(d), ctypes.byref(c), ctypes.byref(r), None, 512, None, 128, None, 128,
                                  A.addr, 0, None, None, 512, None, None)
    assert st == vb.VG_ERR_INVALID_ARG  # (prefix_len has a length of its own)


def ints(*v):
    return torch.tensor(v, dtype=torch.int32)


@pytest.fixture
def no_calls(monkeypatch):
    """What is refused must be refused before the library is called."""
    def call(*args, **kw):
        raise AssertionError("the library was called")
    for name in ("vg_pages_resize", "vg_pages_fork", "vg_pages_compact", "vg_rope_append", "vg_shared_verify_attn"):
        monkeypatch.setattr(vb, name, call)


BAD_LISTS = {
    "int64": torch.tensor([1, 2]),
    "shorter": ints(1),
    "longer": ints(1, 2, 3),
    "two dimensions": ints(1, 2).view(2, 1),
    "apart": ints(1, 0, 2, 0)[::2],
    "elsewhere": torch.empty(2, dtype=torch.int32, device="meta"),
}


@pytest.mark.parametrize("what", list(BAD_LISTS))
def test_request_lists_are_checked(no_calls, what):
    pool, good, bad = make_pool(), ints(1, 2), BAD_LISTS[what]
    with pytest.raises(ValueError):
        pool.resize(bad, good)
    with pytest.raises(ValueError):
        pool.fork(bad, good, good)
    with pytest.raises(ValueError):
        pool.fork(good, bad, good)
    with pytest.raises(ValueError):
        pool.fork(good, good, bad)
    with pytest.raises(ValueError):
        pool.resize(good, bad)
    if what not in ("shorter", "longer"):
        with pytest.raises(ValueError):
            pool.resize(None, bad)


def test_request_lists_that_fit_are_passed_on(monkeypatch):
    pool, seen = make_pool(), []
    monkeypatch.setattr(vb, "vg_pages_resize", lambda *a, **kw: seen.append(a[1:4]))
    monkeypatch.setattr(vb, "vg_pages_fork", lambda *a, **kw: seen.append(a[3:8]))
    a, b, c = ints(3, 4), ints(0, 1), ints(7, 9)
    pool.resize(a, c)
    pool.resize(None, c)
    pool.fork(b, a, c, 5)
    assert seen == [(a, c, 2), (None, c, 2), (b, a, c, 2, 5)]


def layer(slots=48, heads=2, d=64, dtype=torch.bfloat16, device="cpu"):
    return torch.zeros(slots, heads, d, dtype=dtype, device=device)


@pytest.mark.parametrize("K,V", [
    (torch.zeros(48, 2, 2, 64, dtype=torch.bfloat16)[:, 0], layer()),   # K and V of a token side by side
    (layer(), torch.zeros(48, 2, 2, 64, dtype=torch.bfloat16)[:, 1]),
    (layer(heads=4)[:, ::2], layer()),
    (layer(), layer(47)),
    (layer(), layer(heads=1)),
    (layer(), layer(dtype=torch.float32)),
    (layer(), layer(device="meta")),
])
def test_layers_that_are_not_dense_or_not_alike_are_refused(K, V):
    with pytest.raises(ValueError):
        make_pool(kv=[(K, V)])
    with pytest.raises(ValueError):
        make_pool(kv=[(layer(), layer()), (K, V)])
    with pytest.raises(ValueError):
        vb.make_caches([(layer(), layer()), (K, V)])


def test_layers_with_too_few_slots_are_refused_by_the_call():
    pool = make_pool(kv=[(layer(47), layer(47))])
    with pytest.raises(vb.VgError) as e:
        pool.compact(stream=0)
    assert e.value.status == vb.VG_ERR_INVALID_ARG


def test_layers_may_be_slices_of_one_tensor():
    assert len(make_pool(kv=[(layer(), layer().view(48, 128))]).caches) == 1
    kv = torch.zeros(3, 2, 48, 2, 64, dtype=torch.bfloat16)
    pool = make_pool(kv=[(kv[i, 0], kv[i, 1]) for i in range(3)])
    assert len(pool.caches) == 3 and pool.caches[2].V == kv[2, 1].data_ptr() and pool.token_bytes == 256


# ------------------------------------------------------------ a layer's rows
def make_layer(monkeypatch, **kw):
    import synth
    from self_speculative_sparse_gb300.runtime import LayerState
    monkeypatch.setattr(vb, "vg_workspace_size", lambda dims, k: 256)  # (asks the device)
    w = synth.Workload("rows", B=3, Hq=8, Hkv=2, d=64, gamma=1, k=8, n=20, **kw)
    return LayerState(w, w.layer_pool(0), device="cpu")


def row(heads, rows=6, **kw):
    return torch.zeros(rows, heads, 64, dtype=kw.get("dtype", torch.bfloat16), device=kw.get("device", "cpu"))


BAD_ROWS = {
    "fewer rows": lambda h: row(h, rows=5),
    "more rows": lambda h: row(h, rows=7),
    "a row a sequence": lambda h: row(h).view(3, 2, h, 64),
    "one dimension": lambda h: row(h).reshape(-1),
    "fewer heads": lambda h: row(h)[:, :1],
    "more heads": lambda h: row(h + 1),
    "float32": lambda h: row(h, dtype=torch.float32),
    "float16": lambda h: row(h, dtype=torch.float16),
    "elsewhere": lambda h: row(h, device="meta"),
    "heads apart": lambda h: row(2 * h)[:, ::2],
    "elements apart": lambda h: torch.zeros(6, h, 128, dtype=torch.bfloat16)[..., ::2],
    "heads in another order": lambda h: torch.zeros(6, 64, h, dtype=torch.bfloat16).transpose(1, 2),
}


@pytest.mark.parametrize("what", list(BAD_ROWS))
def test_rows_to_rotate_are_checked(no_calls, monkeypatch, what):
    st, rope = make_layer(monkeypatch), vb.vg_rope(A.addr, 64, 0, 1.0)
    good = dict(q=row(8), k=row(2), v=row(2), q_out=row(8))
    for name, t in good.items():
        bad = dict(good, **{name: BAD_ROWS[what](t.shape[1])})
        with pytest.raises(ValueError, match=name):
            st.rope_append(rope, **bad)


def test_rows_that_fit_are_passed_on(monkeypatch):
    st, rope, seen = make_layer(monkeypatch), vb.vg_rope(A.addr, 64, 0, 1.0), []
    monkeypatch.setattr(vb, "vg_rope_append", lambda *a, **kw: seen.append(a[3:]))
    qkv = torch.zeros(6, 12 * 64, dtype=torch.bfloat16)  # slices of one projection's output
    q, k, v = qkv.split((512, 128, 128), 1)
    st.rope_append(rope, q, k, v)
    st.rope_append(rope, q.view(6, 8, 64), k.view(6, 2, 64), v, q_out=row(8))
    assert [x[1] for x in seen] == [768, 768] and [x[7] for x in seen] == [6, 6] and [x[10] for x in seen] == [768, 512]


def test_a_shared_verification_of_two_masks_is_refused(no_calls, monkeypatch):
    st = make_layer(monkeypatch, extra_rows="all")
    assert st.mask1 and st.scores1 is not None
    with pytest.raises(ValueError, match="mask"):
        st.verify_shared(vb.vg_prefix_groups(1, None, A.addr), st.ws)


def test_a_shared_verification_of_one_mask_is_passed_on(monkeypatch):
    st, seen = make_layer(monkeypatch), []
    monkeypatch.setattr(vb, "vg_shared_verify_attn", lambda *a, **kw: seen.append(a))
    st.verify_shared(vb.vg_prefix_groups(1, None, A.addr), st.ws)
    assert len(seen) == 1 and seen[0][7] == st.mask0 and seen[0][8] is st.scores0


# ------------------------------------------------------------ the largest pools
@pytest.mark.parametrize("fits,kw", [
    (True, dict(n_pages=1 << 30, page_size=1)), (False, dict(n_pages=(1 << 30) + 1, page_size=1)),
    (False, dict(n_pages=(1 << 31) - 1, page_size=1)), (True, dict(n_pages=(1 << 30) - 1, page_size=2)),
    (False, dict(n_pages=1 << 30, page_size=2)),
    (True, dict(n_seqs=1, pages_per_seq=1 << 30)), (False, dict(n_seqs=1, pages_per_seq=(1 << 30) + 1)),
    (False, dict(n_seqs=1, pages_per_seq=(1 << 31) - 1)), (False, dict(n_seqs=2, pages_per_seq=1 << 30)),
])
def test_pools_stay_within_what_the_kernels_count_in_32_bits(fits, kw):
    p = vb.vg_page_pool(**{**dict(page_table=A.addr, held=A.addr, refs=A.addr, n_seqs=8, pages_per_seq=16, n_pages=64,
                                  page_size=16), **kw})
    lib = vb.load()
    assert (lib.vg_pages_workspace_size(ctypes.byref(p)) > 0) == fits
    if not fits:
        assert lib.vg_pages_resize(ctypes.byref(p), A.addr, A.addr, 1, A.addr, 1 << 40, None, None) == vb.VG_ERR_INVALID_ARG


# ------------------------------------------------------------ structs made from tensors
def test_groups_have_lists_of_the_right_lengths_and_type():
    g = vb.make_groups(ints(0, 2, 5), ints(7, 9))
    assert g.n_groups == 2 and vb.make_groups(None, ints(4)).n_groups == 1
    assert vb.make_groups(ints(0, 2, 5, 0, 0), ints(7, 9)).n_groups == 2  # (a buffer for more)
    for start, shared in [(ints(0, 5), ints(7, 9)), (ints(), ints()), (torch.tensor([0, 2, 5]), ints(7, 9)), (ints(0, 2, 5), torch.tensor([7, 9])),
                          (ints(0, 0, 2, 0, 5)[::2], ints(7, 9)), (ints(0, 2, 5), ints(7, 0, 9)[::2]),
                          (ints(0, 2, 5), ints(7, 9).view(2, 1))]:
        with pytest.raises(ValueError):
            vb.make_groups(start, shared)


def test_a_rotation_has_all_its_frequencies():
    freq = torch.from_numpy(vb.vg_rope_freqs(64, 10000.0).view("int64"))
    assert vb.make_rope(freq, 64).rot_dim == 64
    assert vb.make_rope(torch.from_numpy(vb.vg_rope_freqs(64, 10000.0)), 64).rot_dim == 64
    for bad, rot in [(freq, 66), (freq[:31], 64), (freq.double(), 64), (freq.to(torch.int32), 64),
                     (torch.zeros(64, dtype=torch.int64)[::2], 64)]:
        with pytest.raises(ValueError):
            vb.make_rope(bad, rot)


def test_a_pool_has_a_count_for_every_row():
    table, held, refs = torch.full((6, 5), -1, dtype=torch.int32), ints(0, 0, 0, 0, 0, 0), ints(0, 0, 0)
    p = vb.make_pages(table, held, refs, 16)
    assert (p.n_seqs, p.pages_per_seq, p.n_pages) == (6, 5, 3)
    for bad in [(table, held[:5], refs), (table.long(), held, refs), (table, held.long(), refs), (table, held, refs.long()),
                (table.t(), held[:5], refs), (table[:, :4], held, refs), (table, held, ints(0, 0, 0, 0)[::2]),
                (table.view(6, 5, 1), held, refs)]:
        with pytest.raises(ValueError):
            vb.make_pages(*bad, 16)


def test_structs_keep_their_tensors():
    import gc
    import weakref
    pool = make_pool()
    c = pool.cache(1)
    refs = [weakref.ref(t) for t in (*pool.layers[1], pool.page_table)]
    del pool
    gc.collect()
    assert [r() is not None for r in refs] == [True] * 3 and c.page_table == refs[2]().data_ptr()
    del c
    gc.collect()
    assert all(r() is None for r in refs)
    t = [torch.zeros(4, 1, 64, dtype=torch.bfloat16), torch.zeros(4, 1, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int64)]
    c = vb.make_cache(*t)
    refs = [weakref.ref(x) for x in t]
    del t
    assert [r().data_ptr() for r in refs] == [c.K, c.V, c.seq_offset]


@pytest.mark.parametrize("base,factor", [(1e300, 1e20), (10000.0, 1e308), (1e-300, 1e-30)])
def test_a_base_that_its_factor_takes_out_of_range_is_refused(base, factor):
    with pytest.raises(vb.VgError) as e:  # (its frequencies would all be zero, or infinite)
        vb.vg_rope_freqs(64, base, vb.VG_ROPE_BASE, factor)
    assert e.value.status == vb.VG_ERR_INVALID_ARG
    if base > 1:
        assert vb.vg_rope_freqs(64, base, vb.VG_ROPE_PLAIN, factor)[0] > 0
