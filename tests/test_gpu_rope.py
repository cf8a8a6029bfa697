"""vg_rope_append on the GPU against the rotation in float64, at the layouts, head shapes,
lengths and row strides where it can go wrong.

Tolerance, from the arithmetic alone: the angle is off by at most 2^-25 of a turn
(2e-7 rad), sincospif by about 2 units of 2^-24, and the two products and their sum by three
roundings of 2^-24 of what goes in: at most 1e-6 * mscale * (|x| + |y|) before the one
rounding to bf16 (half a step: 2^-8 of the value).  Copied elements are equal bit for bit.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from self_speculative_sparse_gb300 import binding as vb  # noqa: E402
from tests.parity import bf16_to_f64  # noqa: E402

pytestmark = pytest.mark.gpu
KINDS = dict(plain=vb.VG_ROPE_PLAIN, linear=vb.VG_ROPE_LINEAR, base=vb.VG_ROPE_BASE, ramp=vb.VG_ROPE_RAMP)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_speculative_sparse_gb300 import build
    build.build()


class Case:
    """Inputs of one call: a fused projection's rows and a cache of the given layout."""

    def __init__(self, rows, pos, Hq=8, Hkv=2, d=64, page=0, rot=64, inter=False, scaling="plain", factor=8.0,
                 mscale=0.0, base=10000.0, pad_rows=0, seed=1, max_len=None, ragged=True):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.rows, self.pos, self.B = rows, pos, len(rows)
        self.Hq, self.Hkv, self.d, self.page, self.rot, self.inter = Hq, Hkv, d, page, rot, inter
        self.mscale = mscale or 1.0
        self.N = sum(rows) + pad_rows
        self.w = (Hq + 2 * Hkv) * d + 16  # a row stride above the heads' own
        self.qkv = torch.randn(max(self.N, 1), self.w, generator=g, device="cuda").to(torch.bfloat16)
        need = [p + r for p, r in zip(pos, rows)]
        if page:
            W = max(1, max(-(-n // page) for n in need))
            first = [p // page for p in pos]
            pages = sum(-(-n // page) - f for n, f in zip(need, first)) + 2
            perm = np.random.default_rng(seed).permutation(pages)
            table, at = np.full((self.B, W), -7, np.int32), 0
            for b in range(self.B):
                for i in range(first[b], -(-need[b] // page)):
                    table[b, i] = perm[at]
                    at += 1
            self.table = torch.from_numpy(table).cuda()
            self.off = None
            slots = pages * page
        else:
            self.off = torch.tensor(np.concatenate([[0], np.cumsum(np.array(need) + 1)[:-1]]), dtype=torch.int64, device="cuda")
            self.table = None
            slots = sum(need) + self.B
        self.K = torch.full((slots, Hkv, d), 3.0, dtype=torch.bfloat16, device="cuda")
        self.V = torch.full((slots, Hkv, d), 5.0, dtype=torch.bfloat16, device="cuda")
        self.row_start = (torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device="cuda")
                          if ragged else None)
        self.prefix = torch.tensor(pos, dtype=torch.int32, device="cuda")
        self.inv = oracle.rope_inverse(rot, base, scaling, factor, 4096.0)
        self.freq = torch.from_numpy(vb.vg_rope_freqs(rot, base, KINDS[scaling], factor, 4096.0).view("int64")).cuda()
        self.rope = vb.make_rope(self.freq, rot, int(inter), mscale)
        gamma = 0 if ragged else rows[0] - 1
        self.dims = vb.make_dims(self.B, Hq, Hkv, d, gamma, max(pos) if max_len is None else max_len)
        self.cache = vb.make_cache(self.K, self.V, self.off, page_table=self.table, page_size=page)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.q_out = torch.full((max(self.N, 1), Hq * d + 8), 9.0, dtype=torch.bfloat16, device="cuda")

    def call(self, in_place=False, stream=None):
        a = self.qkv.data_ptr()
        qd, kd = self.Hq * self.d, self.Hkv * self.d
        vb.vg_rope_append(self.dims, self.cache, self.rope, a, self.w, a + 2 * qd, self.w, a + 2 * (qd + kd), self.w,
                          self.row_start, self.N, self.prefix, a if in_place else self.q_out,
                          self.w if in_place else self.q_out.stride(0), dev_status=self.status, stream=stream)

    def slot(self, b, pos):
        if self.page:
            return int(self.table[b, pos // self.page]) * self.page + pos % self.page
        return int(self.off[b]) + pos

    def check(self, q_out, qkv):
        """q_out: [N][>= Hq d] as called; qkv: the rows before the call."""
        Hq, Hkv, d, rot = self.Hq, self.Hkv, self.d, self.rot
        n = sum(self.rows)
        x = bf16_to_f64(qkv[:n, :(Hq + 2 * Hkv) * d]).reshape(n, Hq + 2 * Hkv, d)
        where = [(b, self.pos[b] + t) for b in range(self.B) for t in range(self.rows[b])]
        pos = np.array([p for _, p in where], dtype=np.int64)
        ref = oracle.rope(x[:, :Hq + Hkv], pos, self.inv, self.inter, self.mscale)
        half = rot // 2
        first = np.arange(half) * (2 if self.inter else 1)
        second = first + (1 if self.inter else half)
        size = np.zeros_like(ref)
        size[..., first] = size[..., second] = np.abs(x[:, :Hq + Hkv, first]) + np.abs(x[:, :Hq + Hkv, second])
        tol = np.abs(ref) * 2.0 ** -8 + 1.01e-6 * self.mscale * size
        got = np.empty_like(ref)
        got[:, :Hq] = bf16_to_f64(q_out[:n, :Hq * d]).reshape(n, Hq, d)
        slots = [self.slot(b, p) for b, p in where]
        K, V = bf16_to_f64(self.K), bf16_to_f64(self.V)
        got[:, Hq:] = K[slots]
        assert (np.abs(got - ref) <= tol).all(), np.abs(got - ref).max()
        assert np.array_equal(got[..., rot:], ref[..., rot:])
        assert np.array_equal(V[slots], x[:, Hq + Hkv:])
        rest = np.setdiff1d(np.arange(K.shape[0]), slots)
        assert (K[rest] == 3.0).all() and (V[rest] == 5.0).all()


SHAPES = [dict(Hq=8, Hkv=2, d=64, rot=64), dict(Hq=32, Hkv=8, d=128, rot=128), dict(Hq=16, Hkv=1, d=64, rot=32),
          dict(Hq=3, Hkv=3, d=128, rot=6), dict(Hq=5, Hkv=1, d=64, rot=2), dict(Hq=4, Hkv=4, d=128, rot=48),
          dict(Hq=2, Hkv=1, d=128, rot=100)]


@pytest.mark.parametrize("page", [0, 1, 5, 16, 64])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_rows_of_a_ragged_batch(shape, inter, page):
    c = Case([1, 0, 7, 130, 0, 3], [0, 5, 63, 1000, 2, 4095], page=page, inter=inter, **SHAPES[shape])
    before = c.qkv.clone()
    c.call()
    torch.cuda.synchronize()
    assert c.status.item() == 0
    c.check(c.q_out, before)
    assert torch.equal(c.qkv, before)
    assert (c.q_out[:, c.Hq * c.d:] == 9.0).all()


@pytest.mark.parametrize("scaling", list(KINDS))
@pytest.mark.parametrize("inter", [False, True])
def test_scalings_at_far_positions(scaling, inter):
    c = Case([4, 4, 4], [65535, 262140, 100000000], Hq=8, Hkv=2, d=128, rot=128, inter=inter, page=16,
             scaling=scaling, factor=32.0, mscale=1.25, base=500000.0)
    before = c.qkv.clone()
    c.call()
    torch.cuda.synchronize()
    assert c.status.item() == 0
    c.check(c.q_out, before)


@pytest.mark.parametrize("B", [1, 31, 33, 300, 1024])
def test_row_lookup_over_many_sequences(B):
    r = np.random.default_rng(B)
    rows = r.integers(0, 4, B).tolist()
    rows[0] = max(rows[0], 1)
    c = Case(rows, r.integers(0, 500, B).tolist(), Hq=2, Hkv=1, d=64, page=16, seed=B)
    before = c.qkv.clone()
    c.call()
    torch.cuda.synchronize()
    assert c.status.item() == 0
    c.check(c.q_out, before)


@pytest.mark.parametrize("rot,inter", [(64, False), (64, True), (6, False)])
def test_in_place_and_uniform_rows_equal_the_packed_call(rot, inter):
    a = Case([4] * 5, [0, 1, 15, 16, 700], rot=rot, inter=inter, page=16, ragged=False)
    b = Case([4] * 5, [0, 1, 15, 16, 700], rot=rot, inter=inter, page=16)
    a.call(in_place=True)
    b.call()
    torch.cuda.synchronize()
    n = a.Hq * a.d
    assert torch.equal(a.qkv[:, :n], b.q_out[:, :n])
    assert torch.equal(a.K, b.K) and torch.equal(a.V, b.V)
    assert torch.equal(a.qkv[:, n:], b.qkv[:, n:])


def test_rows_behind_the_last_sequence_are_left_alone():
    c = Case([3, 2], [10, 20], pad_rows=70, page=16)
    c.qkv[5:] = float("nan")
    before = c.qkv.clone()
    c.call()
    torch.cuda.synchronize()
    assert c.status.item() == 0
    c.check(c.q_out, before)
    assert (c.q_out[5:] == 9.0).all()


def test_many_rows_wrap_around_the_grid():
    c = Case([9000, 5000], [3, 40], Hq=2, Hkv=1, d=64, page=64)
    before = c.qkv.clone()
    c.call()
    torch.cuda.synchronize()
    assert c.status.item() == 0
    c.check(c.q_out, before)


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (64, 32, False), (128, 128, True), (64, 20, True),
                                         (64, 64, False), (128, 100, False), (64, 6, False)])
def test_more_rows_than_one_a_cta(d, rot, inter, page):
    c = Case([1, 700, 0, 3, 513], [7, 63, 4, 0, 2000], Hq=6, Hkv=2, d=d, rot=rot, inter=inter, page=page, pad_rows=9,
             mscale=0.75)
    before = c.qkv.clone()
    c.call()
    torch.cuda.synchronize()
    assert c.status.item() == 0
    c.check(c.q_out, before)
    assert (c.q_out[1217:] == 9.0).all()
    c.call(in_place=True)
    torch.cuda.synchronize()
    n = c.Hq * c.d
    assert torch.equal(c.qkv[:1217, :n], c.q_out[:1217, :n]) and torch.equal(c.qkv[1217:], before[1217:])
    assert torch.equal(c.qkv[:, n:], before[:, n:])


@pytest.mark.parametrize("what", ["prefix", "negative", "page", "table"])
def test_bad_rows_are_reported_and_the_others_served(what):
    c = Case([2, 2, 2], [10, 20, 30], page=16)
    good = Case([2, 2, 2], [10, 20, 30], page=16)
    if what == "prefix":
        c.prefix[1] = c.dims.max_len + 1
    elif what == "negative":
        c.prefix[1] = -1
    elif what == "page":
        c.table[1, 20 // 16] = 10 ** 6
    else:
        c.table[1, 20 // 16] = -1
    c.call()
    good.call()
    torch.cuda.synchronize()
    assert c.status.item() == vb.VG_ERR_DEVICE_BOUNDS
    for r in (0, 1, 4, 5):
        assert torch.equal(c.q_out[r], good.q_out[r])
    if what in ("prefix", "negative"):
        assert (c.q_out[2:4] == 9.0).all()
    else:
        assert torch.equal(c.q_out, good.q_out)
    for b, p in ((0, 10), (0, 11), (2, 30), (2, 31)):
        assert torch.equal(c.K[good.slot(b, p)], good.K[good.slot(b, p)])
    assert (c.K[good.slot(1, 20)] == 3.0).all()


def test_captured_and_replayed_on_another_stream():
    c = Case([4] * 3, [0, 100, 31], page=16)
    s = torch.cuda.Stream()
    c.call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.call()
    for seed in (0, 1):  # the buffers' contents at the replay count
        c.qkv.copy_(torch.randn(c.qkv.shape, generator=torch.Generator().manual_seed(seed)))
        before = c.qkv.clone()
        c.K.fill_(3.0)
        c.V.fill_(5.0)
        g.replay()
        torch.cuda.synchronize()
        c.check(c.q_out, before)
