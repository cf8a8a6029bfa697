"""A batch of branches of one prompt, as a decode loop runs it: the prompt's rows rotated into a
paged cache, branches forked, then rounds of rotate-and-append, shared verification with scores,
selection, a sparse draft step, acceptance, and pages grown, freed, forked again and compacted,
against a simulation that keeps every sequence's tokens by themselves.

What the calls exchange is taken from the device at each step, so that every comparison is of one
call: tables and counts are equal exactly; a cache row is its fp64 rotation rounded once (half a
step: 2^-8 relative) or off by 2^-20 of its pair's length before that rounding, for the fp32 sine,
cosine and products; attention as in the verification's own test (2^-8 (A + 2 |out|) + 2^-14 A,
A = sum_i p_i |v_i|); a draft step's tolerance is the same bound; scores to 2^-18 of the sum of their
products' magnitudes, the selection from them is exact.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from self_speculative_sparse_gb300 import binding as vb  # noqa: E402
from tests.parity import assert_topk_exact, bf16_to_f64  # noqa: E402

pytestmark = pytest.mark.gpu

HQ, HKV, D, GAMMA, PAGE, VOCAB, K_SEL = 8, 2, 64, 3, 16, 50, 40
R = GAMMA + 1
LAYERS = 2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_speculative_sparse_gb300 import build
    build.build()


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def bits(t):
    return t.view(torch.int16)


class Run:
    def __init__(self, rows, pages, seed):
        from self_speculative_sparse_gb300.runtime import PagePool
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.rng = np.random.default_rng(seed)
        nan = lambda: torch.full((pages * PAGE, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.pool = PagePool(rows, 40, pages, PAGE, [(nan(), nan()) for _ in range(LAYERS)])
        self.sim = oracle.Pool(rows, 40, pages, PAGE)
        self.inv = oracle.rope_inverse(D, 500000.0)
        freq = vb.vg_rope_freqs(D, 500000.0)
        self.freq = torch.from_numpy(freq.view(np.int64)).cuda()
        self.rope = vb.make_rope(self.freq, D)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.tokens = [[None] * rows for _ in range(LAYERS)]  # (K, V) of the row's tokens in the cache

    def mk(self, *s):
        return torch.randn(*s, generator=self.g, device="cuda").to(torch.bfloat16)

    def pages_equal(self):
        torch.cuda.synchronize()
        assert self.pool.check_status() == 0 and not self.sim.errors
        table, held = self.pool.page_table.cpu().numpy(), self.pool.held.tolist()
        assert held == [len(r) for r in self.sim.rows] and self.pool.refs.tolist() == self.sim.refs
        for s, r in enumerate(self.sim.rows):
            assert table[s, :len(r)].tolist() == r

    def slots(self, s, n):
        return torch.from_numpy(oracle.paged_slots(self.pool.page_table[s].cpu().numpy(), PAGE, n)).cuda()

    def cache_holds_the_tokens(self, lens):
        """Whatever pages moved or were shared, each row reads its own tokens."""
        for layer, (K, V) in enumerate(self.pool.layers):
            for s, n in enumerate(lens):
                if n == 0:
                    continue
                at = self.slots(s, n)
                k, v = self.tokens[layer][s]
                assert torch.equal(bits(K[at]), bits(k[:n])) and torch.equal(bits(V[at]), bits(v[:n])), (layer, s)

    def append(self, layer, lens, counts):
        """New rows of sequence b, counts[b] of them, behind its first lens[b] tokens; returns the
        rotated queries."""
        N = sum(counts)
        start = np.concatenate([[0], np.cumsum(counts)])
        pad = 3
        qkv = self.mk(N + pad, (HQ + 2 * HKV) * D)
        x = bf16_to_f64(qkv).reshape(N + pad, HQ + 2 * HKV, D)
        q = qkv[:, :HQ * D]
        k, v = qkv[:, HQ * D:(HQ + HKV) * D], qkv[:, (HQ + HKV) * D:]
        q_out = torch.full((N + pad, HQ, D), 7.0, dtype=torch.bfloat16, device="cuda")
        dims = vb.make_dims(len(lens), HQ, HKV, D, GAMMA, 40 * PAGE)
        w = qkv.stride(0)
        vb.vg_rope_append(dims, self.pool.cache(layer), self.rope, q, w, k, w, v, w, ints(start), N + pad,
                          ints(lens), q_out, HQ * D, dev_status=self.status)
        torch.cuda.synchronize()
        assert self.status.item() == 0
        assert (q_out[N:] == 7.0).all()
        pos = np.concatenate([lens[b] + np.arange(c) for b, c in enumerate(counts)])
        want = oracle.rope(x[:N, :HQ + HKV], pos, self.inv, False)
        pair = np.hypot(x[:N, :HQ + HKV, :D // 2], x[:N, :HQ + HKV, D // 2:])
        tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * np.concatenate([pair, pair], -1)
        got_q = bf16_to_f64(q_out[:N])
        assert (np.abs(got_q - want[:, :HQ]) <= tol[:, :HQ]).all()
        K, V = self.pool.layers[layer]
        for b, c in enumerate(counts):
            if c == 0:
                continue
            i = slice(start[b], start[b + 1])
            at = self.slots(b, lens[b] + c)[lens[b]:]
            assert (np.abs(bf16_to_f64(K[at]) - want[i, HQ:]) <= tol[i, HQ:]).all()
            assert torch.equal(bits(V[at]), bits(v[i].reshape(c, HKV, D)))
            old = self.tokens[layer][b]
            both = [K[at].clone(), V[at].clone()]
            if old is not None:
                both = [torch.cat([o[:lens[b]], x]) for o, x in zip(old, both)]
            self.tokens[layer][b] = both
        return q_out[:N]


def attention_close(got, q, K, V, kn, vn):
    ref = oracle.verify_attention(q, K, V, kn, vn)
    A = oracle.verify_attention(q, K, np.abs(V), kn, np.abs(vn))
    tol = 2.0 ** -8 * (A + 2 * np.abs(ref)) + 2.0 ** -14 * A
    assert (np.abs(got - ref) <= tol).all(), np.abs(got - ref).max()


@pytest.mark.parametrize("prompt", [1, 143, 300])
def test_branches_of_a_prompt(prompt):
    B = 6
    run = Run(rows=8, pages=170, seed=prompt)
    pool, sim = run.pool, run.sim
    # the prompt enters the cache through row 0
    room = 40
    pool.resize(None, ints([prompt + room]))
    sim.resize([0], [prompt + room])
    run.pages_equal()
    for layer in range(LAYERS):
        run.append(layer, [0], [prompt])
    # five branches of it, cut at different lengths, all with the first `shared` tokens
    lens = [prompt] + [max(prompt - i, 1) for i in range(B - 1)]
    shared = min(lens)
    pool.fork(ints([0] * (B - 1)), ints(range(1, B)), ints(lens[1:]), room)
    sim.fork([0] * (B - 1), list(range(1, B)), lens[1:], room)
    run.pages_equal()
    for layer in range(LAYERS):
        for s in range(1, B):
            run.tokens[layer][s] = [x[:lens[s]].clone() for x in run.tokens[layer][0]]
    run.cache_holds_the_tokens(lens)
    for step in range(3):
        groups = vb.make_groups(ints([0, B]), ints([shared]))
        max_len = max(lens)
        dims = vb.make_dims(B, HQ, HKV, D, GAMMA, max_len)
        prefix = ints(lens)
        stride = max_len + 5
        for layer in range(LAYERS):
            cache = pool.cache(layer)
            q = run.append(layer, lens, [R] * B).reshape(B, R, HQ, D)
            scores = torch.full((B, stride), 9.0, device="cuda")
            out = torch.empty(B, R, HQ, D, dtype=torch.bfloat16, device="cuda")
            ws = torch.full((vb.vg_shared_verify_workspace_size(dims, groups),), 0xFF, dtype=torch.uint8,
                            device="cuda")
            vb.vg_shared_verify_attn(dims, cache, groups, q, None, None, prefix, 0b1001, scores, stride, out, ws,
                                     dev_status=run.status)
            k_sel = min(K_SEL, max_len)
            idx, count = torch.empty(B, k_sel, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
            vb.vg_topk_select(scores, stride, prefix, B, max_len, k_sel, idx, count, dev_status=run.status)
            # one draft step of another query on the selection; its tail is the first verify row's token
            qd = run.mk(B, HQ, D)
            kd, vd = run.mk(B, HKV, D), run.mk(B, HKV, D)
            od = torch.empty(B, HQ, D, dtype=torch.bfloat16, device="cuda")
            ws2 = torch.empty(vb.vg_workspace_size(dims, k_sel), dtype=torch.uint8, device="cuda")
            vb.vg_sparse_draft_attn(dims, cache, qd, kd, vd, idx, count, k_sel, prefix, ints([1] * B), od, ws2,
                                    dev_status=run.status)
            torch.cuda.synchronize()
            assert run.status.item() == 0
            qf, of, sc = bf16_to_f64(q), bf16_to_f64(out), scores.cpu().numpy()
            for b in range(B):
                n = lens[b]
                k, v = (bf16_to_f64(x) for x in run.tokens[layer][b])
                attention_close(of[b], qf[b], k[:n], v[:n], k[n:n + R], v[n:n + R])
                want = oracle.aggregated_scores(qf[b], k[:n], [0, GAMMA])
                size = np.einsum("hd,nhd->n", np.abs(qf[b][[0, GAMMA]]).reshape(-1, HKV, HQ // HKV, D).sum((0, 2)),
                                 np.abs(k[:n])) / np.sqrt(D)
                assert (np.abs(sc[b, :n] - want) <= 2.0 ** -18 * size).all() and (sc[b, n:] == 9.0).all()
                T = assert_topk_exact(idx[b].cpu().numpy(), int(count[b]), sc[b, :n], k_sel, n, f"selection {b}")
                kt, vt = bf16_to_f64(kd[b:b + 1]), bf16_to_f64(vd[b:b + 1])
                ref = oracle.draft_step(bf16_to_f64(qd[b]), k[:n], v[:n], T, kt, vt)
                A = oracle.draft_step(bf16_to_f64(qd[b]), k[:n], np.abs(v[:n]), T, kt, np.abs(vt))
                assert (np.abs(bf16_to_f64(od[b]) - ref) <= 2.0 ** -8 * (A + 2 * np.abs(ref)) + 2.0 ** -14 * A).all()
                # (the draft step wrote its token where the first verify row's was)
                run.tokens[layer][b][0][n], run.tokens[layer][b][1][n] = kd[b], vd[b]
        # acceptance moves the lengths on
        p_logits = torch.randn(B, R, VOCAB, generator=run.g, device="cuda")
        x = p_logits[:, :GAMMA].argmax(-1).to(torch.int32)
        wrong = run.rng.integers(0, GAMMA + 1, B)
        for b in range(B):
            if wrong[b] < GAMMA:
                x[b, wrong[b]] = (x[b, wrong[b]] + 1) % VOCAB
        acc, nxt = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
        ws3 = torch.empty(vb.vg_accept_workspace_size(B, GAMMA, VOCAB), dtype=torch.uint8, device="cuda")
        vb.vg_accept(B, GAMMA, VOCAB, p_logits, None, x, None, None, vb.VG_ACCEPT_GREEDY, acc, nxt, prefix, ws3,
                     dev_status=run.status)
        torch.cuda.synchronize()
        assert run.status.item() == 0 and acc.tolist() == wrong.tolist()
        lens = [oracle.next_prefix_len(n, int(a)) for n, a in zip(lens, wrong)]
        assert prefix.tolist() == lens
        # pages: cut to what is in use and a step's room, end row 5, branch it again from row 2, close holes
        grow = ints([n + R for n in lens])
        pool.resize(None, grow)
        sim.resize(range(B), [n + R for n in lens])
        pool.resize(ints([5]), ints([0]))
        sim.resize([5], [0])
        pool.fork(ints([2]), ints([5]), ints([lens[2]]), R)
        sim.fork([2], [5], [lens[2]], R)
        pool.compact()
        sim.compact()
        run.pages_equal()
        lens[5] = lens[2]
        for layer in range(LAYERS):
            run.tokens[layer][5] = [t.clone() for t in run.tokens[layer][2]]
        assert pool.n_live.item() == sum(r > 0 for r in sim.refs)
        run.cache_holds_the_tokens(lens)


@pytest.mark.parametrize("page", [0, 16])
def test_a_layers_state_rotates_appends_and_verifies(page):
    import synth
    from self_speculative_sparse_gb300.runtime import LayerState
    w = synth.Workload("branches", B=5, Hq=HQ, Hkv=HKV, d=D, gamma=GAMMA, k=64, n=300)
    data = w.layer_pool(0)
    shared = 261
    o = data["seq_offset"]
    for b in range(1, w.B):
        for x in (data["K"], data["V"]):
            x[o[b]:o[b] + shared] = x[o[0]:o[0] + shared]
    if page:
        data = synth.to_paged(w, data, page)
    st = LayerState(w, data)
    rows = w.B * w.R
    inv = oracle.rope_inverse(D, 10000.0)
    freq = torch.from_numpy(vb.vg_rope_freqs(D, 10000.0).view(np.int64)).cuda()
    q0, k0 = st.q_verify.clone(), st.k_new.clone()
    with pytest.raises(ValueError):
        st.rope_append(vb.make_rope(freq, D), st.q_verify.reshape(rows, HQ, D)[..., ::2], st.k_new, st.v_new)
    st.rope_append(vb.make_rope(freq, D), st.q_verify.view(rows, HQ, D), st.k_new.view(rows, HKV, D),
                   st.v_new.view(rows, HKV, D))
    groups = vb.make_groups(None, ints([shared]))
    ws = torch.empty(vb.vg_shared_verify_workspace_size(st.dims, groups), dtype=torch.uint8, device="cuda")
    st.verify_shared(groups, ws, append=False)
    torch.cuda.synchronize()
    assert st.check_status() == 0
    K, V = bf16_to_f64(st.K), bf16_to_f64(st.V)
    q, out, sc = bf16_to_f64(st.q_verify), bf16_to_f64(st.out_verify), st.scores0.cpu().numpy()
    for b in range(w.B):
        n = int(data["prefix_len"][b])
        at = (oracle.paged_slots(data["page_table"][b], page, n + w.R) if page else o[b] + np.arange(n + w.R))
        pos = n + np.arange(w.R)
        for x0, x in ((bf16_to_f64(q0[b]), q[b]), (bf16_to_f64(k0[b]), K[at[n:]])):
            want = oracle.rope(x0, pos, inv, False)
            pair = np.hypot(x0[..., :D // 2], x0[..., D // 2:])
            assert (np.abs(x - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * np.concatenate([pair, pair], -1)).all()
        assert np.array_equal(V[at[n:]], bf16_to_f64(st.v_new[b]))
        attention_close(out[b], q[b], K[at[:n]], V[at[:n]], K[at[n:]], V[at[n:]])
        want = oracle.aggregated_scores(q[b], K[at[:n]], w.rows("c2"))
        size = np.einsum("hd,nhd->n", np.abs(q[b][w.rows("c2")]).reshape(-1, HKV, HQ // HKV, D).sum((0, 2)),
                         np.abs(K[at[:n]])) / np.sqrt(D)
        assert (np.abs(sc[b, :n] - want) <= 2.0 ** -18 * size).all()
