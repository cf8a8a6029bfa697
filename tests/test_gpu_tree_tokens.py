"""vg_tree_accept where the target has no token for a node, as vg_sample leaves it for a row without any (-1)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import tree as ot  # noqa: E402
from self_speculative_sparse_gb300 import binding as vb  # noqa: E402
from tests.test_gpu_tree_attn import grow, ints  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_speculative_sparse_gb300 import build
    build.build()


def accept(parents, draft, target, prefix=None, layers=None, cache=None):
    B, N = draft.shape
    dims = vb.make_dims(B, 2, 1, 64, 0, 1000)
    if cache is None:
        K = torch.zeros((B * 1100, 1, 64), dtype=torch.bfloat16, device="cuda")
        cache = vb.make_cache(K, K.clone(), torch.arange(B, device="cuda") * 1100)
    prefix = ints([100] * B) if prefix is None else prefix
    path, n, nxt, adv, st = ints(np.zeros((B, N))), ints([7] * B), ints([7] * B), prefix.clone(), ints([0])
    vb.vg_tree_accept(dims, cache, layers, ints(parents), N, None, N, ints(draft), ints(target), prefix, path, n, nxt, adv,
                      dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    return path.cpu().numpy(), n.tolist(), nxt.tolist(), (adv - prefix).tolist()


@pytest.mark.parametrize("none", [-1, -2, -2 ** 31])
def test_a_target_without_a_token_continues_nothing(none):
    """Drafts of rows without tokens are -1 too: equal numbers, and yet no token that both have."""
    parents = np.array([[-1, 0, 1, 2, 2]] * 4)
    draft = np.array([[5, none, 3, 4, none], [5, 2, none, 4, none], [5, 2, 3, none, none], [5, 2, 3, 9, none]])
    target = np.array([[none, 3, 4, none, none], [2, none, 4, none, none], [2, 3, none, none, none], [2, 3, 9, none, none]])
    path, n, nxt, adv = accept(parents, draft, target)
    assert n == [0, 1, 2, 3] and nxt == [none] * 4 and adv == [1, 2, 3, 4]
    assert path.tolist() == [[0, -1, -1, -1, -1], [0, 1, -1, -1, -1], [0, 1, 2, -1, -1], [0, 1, 2, 3, -1]]


def test_walks_among_tokens_and_none():
    """Against the oracle, whose drafts below 0 are made different from every target."""
    r = np.random.default_rng(2)
    B, N = 64, 60
    parents = np.array([grow(r, N) for _ in range(B)])
    draft, target = r.integers(-1, 2, (B, N)), r.integers(-1, 2, (B, N))
    path, n, nxt, _ = accept(parents, draft, target)
    apart = np.where(draft < 0, -100, draft)
    for b in range(B):
        want = ot.walk(parents[b], apart[b], target[b])
        assert path[b].tolist() == want + [-1] * (N - len(want))
        assert (n[b], nxt[b]) == (len(want) - 1, target[b, want[-1]])
