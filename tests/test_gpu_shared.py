"""vg_shared_verify_attn on the GPU against the oracle's attention of each sequence by itself.

Tolerances, from the arithmetic: a softmax weight enters the value product as bf16 (half a
step: 2^-8 of it), its sum being taken over the fp32 weights, so an output is off by at
most 2^-8 A, A = sum_i p_i |v_i|, and by 2^-8 |out| for its own rounding (the bound has
twice that, which a sum over rounded weights would need); fp32
logits, exponentials and sums add less than 2^-14 A.  A score is a sum of products of fp32
queries held in three bf16 parts (2^-24 of each) in fp32 additions, some tens of them one
after another: at most 2^-18 of the sum of the products' magnitudes.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from self_speculative_sparse_gb300 import binding as vb  # noqa: E402
from tests.parity import bf16_to_f64  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_speculative_sparse_gb300 import build
    build.build()


class Case:
    """members: sequences of each group; shared: its shared tokens; private: a list per group."""

    def __init__(self, members, shared, private, Hq=8, Hkv=2, d=64, gamma=0, page=16, scores=True, append=True,
                 scale=0.0, seed=0, heavy=False, max_len=None, mask=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.members, self.shared, self.Hq, self.Hkv, self.d, self.page = members, shared, Hq, Hkv, d, page
        self.R, self.append, self.scale = gamma + 1, append, scale
        self.B = sum(members)
        self.n = [s + x for s, m, p in zip(shared, members, private) for x in p]
        assert len(self.n) == self.B
        R, B = self.R, self.B
        self.tok = []  # physical slot of every token of every sequence
        if page:
            tables, at = [], 0
            b = 0
            for m, s in zip(members, shared):
                common = list(range(at, at + s // page))
                at += len(common)
                for _ in range(m):
                    mine = -(-(self.n[b] + R) // page) - len(common)
                    tables.append(common + list(range(at, at + mine)))
                    at += mine
                    b += 1
            perm = rng.permutation(at + 3)
            W = max(len(t) for t in tables)
            self.table_h = np.full((B, W), -5, np.int32)
            for b, t in enumerate(tables):
                self.table_h[b, :len(t)] = perm[t]
                i = np.arange(self.n[b] + R)
                self.tok.append(self.table_h[b, i // page].astype(np.int64) * page + i % page)
            slots = (at + 3) * page
            self.table, self.off = torch.from_numpy(self.table_h).cuda(), None
        else:
            off = np.concatenate([[0], np.cumsum(np.array(self.n) + R + 2)])
            slots = int(off[-1])
            self.tok = [off[b] + np.arange(self.n[b] + R) for b in range(B)]
            self.table, self.off = None, torch.from_numpy(off[:-1].copy()).cuda()
        nan = float("nan")
        self.K = torch.full((slots, Hkv, d), nan, dtype=torch.bfloat16, device="cuda")
        self.V = torch.full((slots, Hkv, d), nan, dtype=torch.bfloat16, device="cuda")
        u = torch.randn(d, generator=g, device="cuda")
        b = 0
        for m, s in zip(members, shared):
            ks, vs = (torch.randn(s, Hkv, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
            if heavy and s:
                ks[::37] = (u * 1.5).to(torch.bfloat16)
            for _ in range(m):
                t = torch.from_numpy(self.tok[b]).cuda()
                self.K[t[:s]], self.V[t[:s]] = ks, vs
                more = self.n[b] - s
                self.K[t[s:self.n[b]]] = torch.randn(more, Hkv, d, generator=g, device="cuda").to(torch.bfloat16)
                self.V[t[s:self.n[b]]] = torch.randn(more, Hkv, d, generator=g, device="cuda").to(torch.bfloat16)
                b += 1
        mk = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        self.q, self.kn, self.vn = mk(B, R, Hq, d), mk(B, R, Hkv, d), mk(B, R, Hkv, d)
        if heavy:
            self.q += u.to(torch.bfloat16)
        if not append:
            for b in range(B):
                t = torch.from_numpy(self.tok[b][self.n[b]:]).cuda()
                self.K[t], self.V[t] = self.kn[b], self.vn[b]
        self.prefix = torch.tensor(self.n, dtype=torch.int32, device="cuda")
        self.start = torch.tensor(np.concatenate([[0], np.cumsum(members)]), dtype=torch.int32, device="cuda")
        self.shared_len = torch.tensor(shared, dtype=torch.int32, device="cuda")
        self.groups = vb.make_groups(self.start, self.shared_len)
        self.max_len = max(self.n) if max_len is None else max_len
        self.dims = vb.make_dims(B, Hq, Hkv, d, gamma, self.max_len, scale)
        self.cache = vb.make_cache(self.K, self.V, self.off, page_table=self.table, page_size=page)
        self.stride = max(4, self.max_len + 3)
        self.rows = ([0, gamma] if gamma else [0]) if mask is None else mask
        self.mask = sum(1 << t for t in self.rows) if scores else 0
        self.scores = torch.full((B, self.stride), 7.0, device="cuda") if scores else None
        self.out = torch.full((B, R, Hq, d), nan, dtype=torch.bfloat16, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = torch.full((vb.vg_shared_verify_workspace_size(self.dims, self.groups),), 0xFF, dtype=torch.uint8,
                             device="cuda")

    def call(self, stream=None):
        vb.vg_shared_verify_attn(self.dims, self.cache, self.groups, self.q, self.kn if self.append else None,
                                 self.vn if self.append else None, self.prefix, self.mask, self.scores, self.stride,
                                 self.out, self.ws, dev_status=self.status, stream=stream)

    def check(self, skip=(), status=0, K0=None, V0=None):
        torch.cuda.synchronize()
        assert self.status.item() == status
        K0 = self.K if K0 is None else K0
        V0 = self.V if V0 is None else V0
        Kc, Vc, out = bf16_to_f64(K0), bf16_to_f64(V0), bf16_to_f64(self.out)
        q, kn, vn = bf16_to_f64(self.q), bf16_to_f64(self.kn), bf16_to_f64(self.vn)
        scale = self.scale or 1.0 / np.sqrt(self.d)
        for b in range(self.B):
            if b in skip:
                continue
            n, t = self.n[b], self.tok[b]
            K, V = Kc[t[:n]], Vc[t[:n]]
            ref = oracle.verify_attention(q[b], K, V, kn[b], vn[b], scale)
            A = oracle.verify_attention(q[b], K, np.abs(V), kn[b], np.abs(vn[b]), scale)
            tol = 2.0 ** -8 * (A + 2 * np.abs(ref)) + 2.0 ** -14 * A
            err = np.abs(out[b] - ref)
            assert (err <= tol).all(), (b, n, err.max(), np.unravel_index(np.nanargmax(err - tol), err.shape))
            if self.mask:
                got = self.scores[b].cpu().numpy().astype(np.float64)
                want = oracle.aggregated_scores(q[b], K, self.rows, scale) if n else np.zeros(0)
                G = self.Hq // self.Hkv
                Q = np.abs(q[b][self.rows].reshape(-1, self.Hkv, G, self.d)).sum((0, 2))
                size = scale * np.einsum("hd,nhd->n", Q, np.abs(K))
                assert (np.abs(got[:n] - want) <= 2.0 ** -18 * size).all(), (b, np.abs(got[:n] - want).max())
                assert (got[n:] == 7.0).all()
            if self.append:
                at = torch.from_numpy(t[n:]).cuda()
                assert torch.equal(self.K[at], self.kn[b]) and torch.equal(self.V[at], self.vn[b])


SMALL = {
    "one_sequence_one_tile": dict(members=[1], shared=[128], private=[[0]]),
    "one_token_prefix": dict(members=[1], shared=[1], private=[[0]]),
    "empty_prefix": dict(members=[2], shared=[0], private=[[0, 0]]),
    "nothing_shared": dict(members=[3], shared=[0], private=[[1, 200, 63]]),
    "below_a_tile": dict(members=[2], shared=[127], private=[[0, 3]]),
    "past_a_tile": dict(members=[2], shared=[129], private=[[0, 300]]),
    "two_groups": dict(members=[2, 3], shared=[300, 513], private=[[5, 0], [1, 130, 2]], gamma=3),
    "group_of_one_and_empty_group": dict(members=[1, 0, 2], shared=[256, 99, 128], private=[[7], [], [0, 1]], gamma=1),
    "odd_kv_heads": dict(members=[5], shared=[400], private=[[3, 0, 9, 128, 256]], Hq=12, Hkv=3, d=128, gamma=2),
    "one_kv_head_16": dict(members=[4], shared=[640], private=[[1, 2, 3, 129]], Hq=16, Hkv=1, d=64, gamma=3),
    "one_row_tile_and_a_row": dict(members=[33], shared=[257], private=[list(range(33))], Hq=8, Hkv=2, d=64, gamma=0),
    "two_row_tiles": dict(members=[8], shared=[384], private=[[2] * 8], Hq=8, Hkv=2, d=128, gamma=7),
    "three_row_tiles": dict(members=[10], shared=[384], private=[[i for i in range(10)]], Hq=8, Hkv=2, d=128, gamma=7),
    "many_row_tiles": dict(members=[40], shared=[512], private=[[i % 5 for i in range(40)]], Hq=16, Hkv=4, d=64, gamma=9),
    "64_rows": dict(members=[3], shared=[200], private=[[70, 1, 0]], Hq=4, Hkv=1, d=128, gamma=15),
    "more_than_64_members": dict(members=[70], shared=[300], private=[[i % 3 for i in range(70)]], Hq=2, Hkv=2, d=64),
    "many_small_groups": dict(members=[1] * 40, shared=[130 + i for i in range(40)], private=[[i] for i in range(40)],
                              Hq=4, Hkv=2, d=64, gamma=1),
    "tall_scale": dict(members=[3], shared=[500], private=[[9, 10, 11]], scale=0.9, gamma=1),
    "peaked": dict(members=[6], shared=[1000], private=[[9, 10, 11, 0, 1, 2]], heavy=True, gamma=2, scale=0.5),
}


@pytest.mark.parametrize("page", [0, 8, 16, 32, 64, 128])
@pytest.mark.parametrize("name", list(SMALL))
def test_matches_each_sequence_by_itself(name, page):
    c = Case(page=page, **SMALL[name])
    K0, V0 = c.K.clone(), c.V.clone()
    c.call()
    c.check(K0=K0, V0=V0)
    # nothing but the verify rows entered the cache
    seen = np.concatenate([t[n:] for t, n in zip(c.tok, c.n)])
    rest = torch.from_numpy(np.setdiff1d(np.arange(c.K.shape[0]), seen)).cuda()
    assert torch.equal(c.K[rest].view(torch.int16), K0[rest].view(torch.int16))
    assert torch.equal(c.V[rest].view(torch.int16), V0[rest].view(torch.int16))


LONG = {
    "heads_mode": dict(members=[16], shared=[20000], private=[[1 + 31 * i for i in range(16)]], Hq=32, Hkv=8, d=128),
    "pair_mode": dict(members=[12, 4], shared=[9000, 5000], private=[[40 * i for i in range(12)], [0, 1, 2, 1500]],
                      Hq=32, Hkv=8, d=128, gamma=6),
    "d64": dict(members=[20], shared=[12345], private=[[i for i in range(20)]], Hq=64, Hkv=8, d=64, gamma=3),
    "long_private": dict(members=[2], shared=[130], private=[[9000, 4000]], Hq=32, Hkv=8, d=128, gamma=7),
    "heavy": dict(members=[9], shared=[15000], private=[[i for i in range(9)]], Hq=16, Hkv=4, d=128, gamma=5, heavy=True),
}


@pytest.mark.parametrize("name", list(LONG))
def test_long_prefixes(name):
    c = Case(page=16 if name != "d64" else 64, **LONG[name])
    K0, V0 = c.K.clone(), c.V.clone()
    c.call()
    c.check(K0=K0, V0=V0)


@pytest.mark.parametrize("gamma", [0, 4])
def test_rows_already_in_the_cache_and_no_scores(gamma):
    c = Case([3, 2], [300, 40], [[1, 2, 300], [0, 5]], gamma=gamma, append=False, scores=False)
    K0 = c.K.clone()
    c.call()
    c.check()
    assert torch.equal(c.K.view(torch.int16), K0.view(torch.int16))


@pytest.mark.parametrize("mask", [[0], [3], [1, 2], [0, 1, 2, 3]])
def test_score_rows(mask):
    c = Case([4], [400], [[0, 3, 130, 9]], gamma=3, mask=mask)
    K0, V0 = c.K.clone(), c.V.clone()
    c.call()
    c.check(K0=K0, V0=V0)


def test_one_group_needs_no_list():
    a, b = (Case([5], [700], [[1, 2, 3, 4, 5]], gamma=2) for _ in range(2))
    b.groups = vb.make_groups(None, b.shared_len)
    a.call()
    b.call()
    torch.cuda.synchronize()
    assert torch.equal(a.out.view(torch.int16), b.out.view(torch.int16)) and torch.equal(a.scores, b.scores)


def test_the_same_call_gives_the_same_bits_and_any_split_of_a_prefix_the_same_values():
    ref = None
    for shared in (0, 130, 900, 1000):
        c = Case([6], [1000], [[0, 1, 2, 30, 40, 500]], gamma=3, append=False)
        c.shared_len.fill_(shared)
        c.call()
        c.check()
        first = c.out.clone()
        c.ws.fill_(0)
        c.call()
        torch.cuda.synchronize()
        assert torch.equal(first.view(torch.int16), c.out.view(torch.int16))
        s = c.scores.clone()
        ref = s if ref is None else ref
        assert torch.equal(s, ref)


@pytest.mark.parametrize("what", ["shared_too_long", "shared_negative", "start_not_zero", "start_descending",
                                  "start_short", "start_far"])
def test_bad_groups_are_reported_and_every_sequence_read_by_itself(what):
    c = Case([2, 3], [300, 513], [[5, 0], [1, 130, 2]], gamma=3)
    K0, V0 = c.K.clone(), c.V.clone()
    if what == "shared_too_long":
        c.shared_len[0] = 301
    elif what == "shared_negative":
        c.shared_len[1] = -1
    elif what == "start_not_zero":
        c.start[0] = 1
    elif what == "start_descending":
        c.start[1] = 6
    elif what == "start_short":
        c.start[2] = 4
    else:
        c.start[2] = 1 << 30
    c.call()
    c.check(status=vb.VG_ERR_DEVICE_BOUNDS, K0=K0, V0=V0)


@pytest.mark.parametrize("who", [0, 1, 3])
@pytest.mark.parametrize("value", [-1, 1 << 20])
def test_a_bad_length_is_reported_and_the_others_are_served(who, value):
    c = Case([2, 3], [300, 513], [[5, 0], [1, 130, 2]], gamma=1)
    K0, V0 = c.K.clone(), c.V.clone()
    c.prefix[who] = value
    c.call()
    c.check(skip=[who], status=vb.VG_ERR_DEVICE_BOUNDS, K0=K0, V0=V0)
    assert torch.isnan(c.out[who]).all()


def test_a_bad_page_of_one_sequence_is_reported_and_the_others_are_served():
    for bad in (-1, 10 ** 6):
        c = Case([3], [256], [[40, 50, 60]], gamma=1, scores=False)
        K0, V0 = c.K.clone(), c.V.clone()
        c.table[1, 256 // 16] = bad
        c.call()
        torch.cuda.synchronize()
        assert c.status.item() == vb.VG_ERR_DEVICE_BOUNDS
        c.check(skip=[1], status=vb.VG_ERR_DEVICE_BOUNDS, K0=K0, V0=V0)


def test_captured_and_replayed_with_other_lengths_on_another_stream():
    c = Case([4, 2], [600, 260], [[0, 10, 200, 300], [5, 600]], gamma=2, append=False)
    c.call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.call()
    n0 = list(c.n)
    for cut in (0, 3):
        # shorter prefixes: the rows behind them are then the tokens that were there
        c.n = [n - cut for n in n0]
        lens = [min(c.n[:4]), min(c.n[4:])]
        c.prefix.copy_(torch.tensor(c.n))
        c.shared_len.copy_(torch.tensor([min(600, lens[0]), min(260, lens[1])]))
        for b in range(c.B):
            t = torch.from_numpy(c.tok[b][c.n[b]:c.n[b] + c.R]).cuda()
            c.kn[b], c.vn[b] = c.K[t], c.V[t]
        c.scores.fill_(7.0)
        c.out.fill_(float("nan"))
        g.replay()
        c.check()


@pytest.mark.parametrize("scores", [False, True])
def test_many_sequences_and_many_runs_of_a_cta(scores):
    # 1024 sequences: every CTA works on a dozen items or more, most of them one or two tiles long
    lens = [(37 * i) % 150 for i in range(1024)]
    c = Case([1000, 24], [200, 130], [lens[:1000], lens[1000:]], Hq=4, Hkv=4, d=64, page=8, scores=scores)
    K0, V0 = c.K.clone(), c.V.clone()
    c.call()
    c.check(K0=K0, V0=V0)


def test_as_many_groups_as_sequences():
    def case(d):
        return Case([1] * 1024, [130] * 1024, [[i % 3] for i in range(1024)], Hq=2, Hkv=1, d=d, page=16)
    c = case(64)
    K0, V0 = c.K.clone(), c.V.clone()
    c.call()
    c.check(K0=K0, V0=V0)
    with pytest.raises(vb.VgError) as e:  # the layout does not fit beside four tiles of 128 columns
        case(128).call()
    assert e.value.status == vb.VG_ERR_UNSUPPORTED_SHAPE


def test_two_captured_calls_share_a_workspace():
    a = Case([4, 2], [600, 260], [[0, 10, 200, 300], [5, 600]], gamma=2, append=False, seed=1)
    b = Case([7], [1000], [[i * 31 for i in range(7)]], gamma=1, append=False, seed=2, scores=False, d=64)
    if b.ws.numel() > a.ws.numel():
        a.ws = b.ws
    else:
        b.ws = a.ws
    graphs = []
    for c in (a, b):
        c.call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call()
        graphs.append(g)
    for c in (a, b):
        c.out.fill_(float("nan"))
        if c.scores is not None:
            c.scores.fill_(7.0)
    for _ in range(3):
        for g in graphs:
            g.replay()
    a.check()
    b.check()


def test_beside_the_verify_call_it_stands_for():
    c = Case([5], [1500], [[0, 7, 64, 100, 333]], Hq=32, Hkv=8, d=128, gamma=4, append=False)
    ws = torch.empty(vb.vg_workspace_size(c.dims, 16), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c.out)
    stride = (c.max_len + 3) // 4 * 4
    sc = torch.full((c.B, stride), 7.0, device="cuda")
    vb.vg_verify_attn(c.dims, c.cache, c.q, None, None, c.prefix, c.mask, 0, sc, None, stride, out, ws,
                      dev_status=c.status)
    c.call()
    torch.cuda.synchronize()
    assert c.status.item() == 0
    assert (c.out.float() - out.float()).abs().max() <= 2.0 ** -5
    for b, n in enumerate(c.n):
        assert (c.scores[b, :n] - sc[b, :n]).abs().max() <= 1e-3 * sc[b, :n].abs().max()
