"""vg_tree_verify_attn where batches are large: more units than two an SM (a CTA then takes several whole ranges in turn), and
the ring of four tiles that is left beside the layout of many sequences at d = 128.  Reference and tolerance as in
test_gpu_tree_attn.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_tree_attn import Tree  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_speculative_sparse_gb300 import build
    build.build()


@pytest.mark.parametrize("scores", [True, False])
@pytest.mark.parametrize("N,Hq,Hkv,d", [(256, 32, 8, 128), (250, 24, 12, 64), (150, 48, 3, 128)])
def test_more_units_of_several_row_tiles_than_two_an_sm(N, Hq, Hkv, d, scores):
    r = np.random.default_rng(N)
    B = 16 if Hkv > 3 else 24
    pre = [int(np.exp(r.uniform(0, 7.2))) for _ in range(B)]
    pre[3], pre[5] = 0, 1500
    lens = [int(r.integers(N // 2, N + 1)) for _ in range(B)]
    lens[0], lens[7], lens[9] = N, 0, 1
    tiles = [-(-m * (Hq // Hkv) // (128 // (Hq // Hkv) * (Hq // Hkv))) for m in lens]
    units = sum(Hkv * (t // 2) + t % 2 * -(-Hkv // 2) for t in tiles)
    assert max(tiles) > 2 and units > (2 * torch.cuda.get_device_properties(0).multi_processor_count if Hkv == 8 else 100)
    Tree(pre, lens, N, Hq, Hkv, d, page=16 if scores else 0, seed=N, scores=scores, fresh=scores).call().check()


@pytest.mark.parametrize("scores", [True, False])
@pytest.mark.parametrize("B,N,Hq,Hkv", [(250, 9, 32, 8), (250, 33, 32, 8), (200, 70, 12, 3), (300, 17, 64, 8), (1000, 5, 6, 3)])
def test_many_sequences_beside_a_ring_of_four_tiles(B, N, Hq, Hkv, scores):
    r = np.random.default_rng(B + N)
    pre = r.integers(0, 900, B).tolist()
    lens = r.integers(0, N + 1, B).tolist()
    pre[B // 2], lens[B // 2] = 5000, N
    Tree(pre, lens, N, Hq, Hkv, 128, page=64 if scores else 16, seed=B, scores=scores).call().check()


@pytest.mark.parametrize("B,N", [(250, 9), (200, 70)])
def test_repeated_calls_of_many_sequences_are_bit_identical(B, N):
    r = np.random.default_rng(B)
    c = Tree(r.integers(0, 1200, B).tolist(), r.integers(0, N + 1, B).tolist(), N, 32, 8, 128, page=16, seed=B).call()
    out, scores = c.out.clone(), c.scores.clone()
    for _ in range(20):
        c.out.fill_(9.0)
        c.ws.view(torch.float32).fill_(float("inf"))
        c.call()
        assert torch.equal(c.out, out) and torch.equal(c.scores, scores) and c.status.item() == 0
