"""Calls of the batch operators that run at the same time: two streams, each with its own buffers and workspace, give
what the same calls give one after another."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_pages import Both, ints  # noqa: E402
from tests.test_gpu_rope import Case as RopeCase  # noqa: E402
from tests.test_gpu_shared import Case as SharedCase  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_speculative_sparse_gb300 import build
    build.build()


def make(seed):
    """A shared verification, a rotary append and a pool of its own, and a step of them on a stream."""
    shared = SharedCase([6, 3], [1200, 700], [[0, 10, 200, 300, 31, 5], [5, 600, 77]], gamma=2, append=False, seed=seed,
                        Hq=16, Hkv=4, d=128 if seed % 2 else 64)
    rope = RopeCase([3, 700, 2], [10, 20, 300], page=16, seed=seed)
    pool = Both(40, 12, 200, 8, layers=2, seed=seed).gpu
    seq, length = ints([1, 2, 3, 0]), ints([40 + seed, 17, 60, 33])
    parent, child, part = ints([1, 3, 3]), ints([10, 11, 12]), ints([25, 41, 60])

    def step(stream):
        shared.call(stream=stream)
        rope.call(stream=stream)
        pool.resize(seq, length, stream=stream)
        pool.fork(parent, child, part, 9, stream=stream)
        pool.resize(ints_two, ints_zero, stream=stream)
        pool.compact(stream=stream)

    ints_two, ints_zero = ints([2]), ints([0])
    out = lambda: [shared.out, shared.scores, rope.q_out, rope.K, rope.V, pool.page_table, pool.held, pool.refs,  # noqa: E731
                   pool.n_live, shared.status, rope.status, pool.status] + [t for kv in pool.layers for t in kv]
    return step, out


def bits(ts):
    return [t.view(torch.int16).clone() if t.dtype == torch.bfloat16 else t.clone() for t in ts]


def test_two_streams_at_once():
    want = []
    for seed in (1, 2):
        step, out = make(seed)
        for _ in range(8):
            step(torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append(bits(out()))
        assert out()[9].item() == out()[10].item() == out()[11].item() == 0
    both = [make(seed) for seed in (1, 2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(8):
        for (step, _out), s in zip(both, streams):
            step(s)
    torch.cuda.synchronize()
    for (_step, out), w in zip(both, want):
        for a, b in zip(bits(out()), w):
            assert torch.equal(a, b)
