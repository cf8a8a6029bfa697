"""The page pool's calls on the GPU against the list simulation, step after step on one pool:
tables, counts, references and the contents of every layer are equal exactly, and so is what
is refused."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from self_speculative_sparse_gb300 import binding as vb  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_speculative_sparse_gb300 import build
    build.build()


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


class Both:
    """A PagePool on the GPU and the simulation beside it, with the same contents."""

    def __init__(self, n_seqs, pages_per_seq, n_pages, page, layers=1, heads=(1, 8), seed=0):
        from self_speculative_sparse_gb300.runtime import PagePool
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        H, d = heads
        mk = lambda: torch.randint(-30000, 30000, (n_pages * page, H, d), generator=g, device="cuda").to(torch.int16).view(torch.bfloat16)  # noqa: E731
        self.gpu = PagePool(n_seqs, pages_per_seq, n_pages, page, [(mk(), mk()) for _ in range(layers)])
        self.gpu.ws.fill_(0xA5)
        self.sim = oracle.Pool(n_seqs, pages_per_seq, n_pages, page)
        self.data = [t.view(torch.int16).cpu().numpy().copy() for kv in self.gpu.layers for t in kv]
        self.page = page

    def _move(self, src, dst, tokens):
        for t in self.data:
            t[dst * self.page:dst * self.page + tokens] = t[src * self.page:src * self.page + tokens]

    def resize(self, seq, length, stream=None):
        if len(length):
            self.gpu.resize(None if seq is None else ints(seq), ints(length), stream=stream)
        self.sim.resize(range(len(length)) if seq is None else seq, length)
        self.check()

    def fork(self, parent, child, length, room=0):
        if len(length):
            self.gpu.fork(ints(parent), ints(child), ints(length), room)
        for c in self.sim.fork(parent, child, length, room):
            self._move(*c)
        self.check()

    def compact(self):
        self.gpu.compact()
        for src, dst in self.sim.compact():
            self._move(src, dst, self.page)
        self.check()
        assert self.gpu.n_live.item() == sum(r > 0 for r in self.sim.refs)

    def check(self):
        torch.cuda.synchronize()
        table, held = self.gpu.page_table.cpu().numpy(), self.gpu.held.cpu().numpy()
        assert held.tolist() == [len(r) for r in self.sim.rows]
        for s, r in enumerate(self.sim.rows):
            assert table[s, :len(r)].tolist() == r, s
            assert (table[s, len(r):] == -1).all(), s
        assert self.gpu.refs.cpu().tolist() == self.sim.refs
        for t, want in zip([t for kv in self.gpu.layers for t in kv], self.data):
            assert np.array_equal(t.view(torch.int16).cpu().numpy(), want)
        want = self.sim.errors[:1]
        got = self.gpu.check_status()
        assert got in ({"bounds": [vb.VG_ERR_DEVICE_BOUNDS], "pages": [vb.VG_ERR_DEVICE_PAGES]}[want[0]] if len(set(self.sim.errors)) == 1
                       else [vb.VG_ERR_DEVICE_BOUNDS, vb.VG_ERR_DEVICE_PAGES]) if want else got == 0
        self.gpu.status.zero_()
        self.sim.errors.clear()


@pytest.mark.parametrize("page", [1, 5, 16, 64])
def test_a_life_of_requests(page):
    p = Both(12, 40, 300, page, layers=2, heads=(2, 8))
    r = np.random.default_rng(page)
    p.resize(None, (r.integers(0, 20, 8) * page + r.integers(0, 2, 8)).tolist())
    for _ in range(6):
        lens = [len(x) * page for x in p.sim.rows]
        parents = [s for s in range(4)]
        f = r.choice(parents, 5).tolist()
        c = r.permutation(np.arange(4, 12))[:5].tolist()
        p.fork(f, c, [int(r.integers(0, lens[x] + 1)) for x in f], int(r.integers(0, 9)))
        s = r.permutation(12)[:6].tolist()
        p.resize(s, [int(r.integers(0, 25 * page)) for _ in s])
        p.compact()


def test_zero_and_one():
    p = Both(3, 2, 4, 16)
    p.resize([0], [0])
    p.resize([0], [1])
    p.fork([0], [1], [0], 0)        # an empty branch
    p.fork([0], [1], [1], 0)        # one copied token
    p.fork([1], [2], [1], 15)       # room that fits the copied page
    p.fork([1], [2], [1], 16)       # room for a second page
    p.resize(None, [0, 0, 0])
    p.compact()                     # nothing lives
    assert p.gpu.n_live.item() == 0


def test_a_full_pool_moves_nothing_and_hands_out_nothing():
    p = Both(4, 8, 8, 8)
    p.resize([0, 1], [32, 32])
    p.compact()
    p.resize([2], [1])              # none left
    p.resize([0, 2], [8, 24])       # what one row gives back in the same call
    p.resize([1, 2, 3], [40, 25, 1])  # the first that does not fit stops all later ones


def test_a_fork_that_runs_out_leaves_the_child_empty_and_the_parent_whole():
    p = Both(4, 8, 6, 8)
    p.resize([0, 1], [12, 16])
    p.fork([0, 0], [1, 2], [12, 12], 24)
    p.fork([0], [3], [9], 100)      # longer than a row


def test_refused_requests_change_nothing_and_the_others_are_served():
    p = Both(6, 4, 30, 8)
    p.resize([0, 1], [20, 9])
    p.resize([2, 6, -1, 3], [8, 8, 8, 8])              # rows outside the table
    p.resize([4, 4, 5], [8, 16, 8])                    # named twice: the first counts
    p.resize([4, 5], [-1, 33])                         # negative, longer than a row
    p.fork([0, 9, 0], [2, 3, -4], [10, 1, 2])
    p.fork([0, 2], [2, 3], [10, 5])                    # a parent that is a child too
    p.fork([1, 1], [5, 5], [9, 3])                     # a child named twice
    p.fork([1, 0], [4, 5], [17, 3])                    # longer than the parent holds


def test_a_page_that_is_never_handed_out():
    p = Both(3, 8, 10, 8)
    for i in (0, 5):
        p.sim.refs[i] = 1
        p.gpu.refs[i] = 1
    p.resize(None, [30, 20, 0])
    p.resize([0], [0])
    p.compact()


@pytest.mark.parametrize("n_pages", [3, 4097, 8192, 8193, 40000, 131072, 300001])
def test_pools_that_need_more_than_one_cta(n_pages):
    per = min(n_pages, 500)
    p = Both(600, per, n_pages, 1, heads=(1, 8), seed=3)
    r = np.random.default_rng(n_pages)
    p.resize(None, r.integers(0, max(2, min(per, 2 * n_pages // 700)), 600).tolist())
    s = r.permutation(600)[:400].tolist()
    p.resize(s, [0 if i % 3 == 0 else int(r.integers(0, max(2, min(per, 2 * n_pages // 700)))) for i in range(400)])
    p.compact()


def test_one_parent_of_many_and_many_layers():
    p = Both(200, 5, 600, 16, layers=5, heads=(2, 64))
    p.resize([0, 1], [70, 33])
    p.fork([0] * 150 + [1] * 40, list(range(2, 192)), [70] * 75 + [64] * 75 + [33] * 40, 3)
    p.resize(list(range(2, 192, 2)), [0] * 95)
    p.compact()


def test_more_requests_than_threads():
    p = Both(5000, 3, 9000, 2, heads=(1, 8))
    p.resize(None, [i % 4 for i in range(5000)])
    p.fork([1] * 2000, list(range(3000, 5000)), [1] * 2000, 1)
    p.resize(list(range(4999, -1, -1)), [i % 3 for i in range(5000)])


def test_pages_larger_than_a_copy_piece():
    p = Both(3, 4, 10, 200, heads=(2, 64))
    p.resize([0], [555])
    p.fork([0, 0], [1, 2], [555, 401], 7)
    p.resize([0], [0])
    p.compact()


def test_outputs_apart_from_the_pool_leave_it_as_it_was():
    p = Both(6, 6, 40, 8, layers=2)
    p.resize(None, [40, 30, 20, 10, 48, 5])
    p.resize([0, 2], [0, 3])
    g = p.gpu
    table, refs, held = g.page_table.clone(), g.refs.clone(), g.held.clone()
    t2, r2 = torch.full_like(table, 77), torch.full_like(refs, 77)
    for _ in range(2):  # the pool stays as it was, so the same call gives the same again
        vb.vg_pages_compact(g.pool, g.caches, g.token_bytes, t2, r2, g.n_live, g.ws, dev_status=g.status)
        torch.cuda.synchronize()
        assert torch.equal(g.page_table, table) and torch.equal(g.refs, refs) and torch.equal(g.held, held)
        sim = oracle.Pool(6, 6, 40, 8)
        sim.rows, sim.refs = [list(x) for x in p.sim.rows], list(p.sim.refs)
        for src, dst in sim.compact():
            p._move(src, dst, 8)
        assert r2.tolist() == sim.refs
        for s, x in enumerate(sim.rows):
            assert t2[s].tolist() == x + table[s, len(x):].tolist()
    p.check()


def test_bad_table_entries_are_reported():
    p = Both(3, 4, 10, 8)
    p.resize(None, [20, 8, 8])
    p.gpu.page_table[0, 1] = 99
    p.gpu.compact()
    torch.cuda.synchronize()
    assert p.gpu.check_status() == vb.VG_ERR_DEVICE_BOUNDS and p.gpu.page_table[0, 1].item() == 99
    p.gpu.status.zero_()
    p.gpu.resize(ints([0]), ints([0]))
    torch.cuda.synchronize()
    assert p.gpu.check_status() == vb.VG_ERR_DEVICE_BOUNDS
    assert p.gpu.held.tolist() == [0, 1, 1] and p.gpu.refs.tolist()[:6] == [0, 1, 0, 1, 1, 0]


def test_captured_calls_replay_on_the_state_they_find():
    p = Both(8, 6, 60, 8)
    seq, length = ints([0, 1, 2]), ints([40, 17, 8])
    f, c, n = ints([0, 0]), ints([4, 5]), ints([13, 24])
    p.gpu.resize(seq, length)   # (loads the kernels before the capture)
    p.gpu.fork(f, c, n, 5)
    p.gpu.compact()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.gpu.resize(seq, length)
        p.gpu.fork(f, c, n, 5)
        p.gpu.compact()
    p = p  # the first calls above changed the pool: start both sides afresh
    p.gpu.page_table.fill_(-1)
    p.gpu.held.zero_()
    p.gpu.refs.zero_()
    p.data = [t.view(torch.int16).cpu().numpy().copy() for kv in p.gpu.layers for t in kv]
    for lens, forks in (([40, 17, 8], [13, 24]), ([3, 0, 33], [1, 3])):
        length.copy_(ints(lens))
        n.copy_(ints(forks))
        g.replay()
        p.sim.resize([0, 1, 2], lens)
        for x in p.sim.fork([0, 0], [4, 5], forks, 5):
            p._move(*x)
        for src, dst in p.sim.compact():
            p._move(src, dst, 8)
        p.check()
