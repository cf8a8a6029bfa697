"""Compaction of a pool that is small beside its table: the table is rewritten by the whole GPU, however few pages
move."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_pages import Both  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_speculative_sparse_gb300 import build
    build.build()


@pytest.mark.parametrize("n_pages", [1, 2, 5])
def test_a_large_table_of_a_small_pool(n_pages):
    p = Both(60000, 64, n_pages, 1)
    rows = [59999, 3][:n_pages]
    p.resize(rows, [1] * len(rows))
    p.resize(rows[:1], [0])      # a hole in front, if there are two rows
    p.compact()
    p.resize([17], [1])
    p.compact()
    # 3.8 million entries, 15 MB read and written: 24 us a call, 4.2 ms by one CTA (a grid made for one
    # page).  The best of five calls has to be far from the second
    best = float("inf")
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        p.gpu.compact()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    assert best < 0.5, f"{best} ms"
