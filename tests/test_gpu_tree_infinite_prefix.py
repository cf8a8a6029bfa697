"""vg_tree_verify_attn over prefixes with keys of infinite values: a logit of -inf has no weight, wherever the key stands (at the
front of a sequence, over whole tiles, where a run of the kernel begins).  The result is attention over the other keys, within
the tolerance of test_gpu_tree_attn.py (which counts tokens, so that the number of weights' bits is the same)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.parity import bf16_to_f64  # noqa: E402
from tests.test_gpu_tree_attn import Tree, attention, ints  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_speculative_sparse_gb300 import build
    build.build()


@pytest.mark.parametrize("shape,N", [((8, 2, 64), 9), ((32, 8, 128), 40), ((48, 3, 128), 20)])
@pytest.mark.parametrize("pre,first,last", [(700, 0, 128), (700, 0, 700), (300, 128, 300), (9000, 0, 128), (9000, 0, 8990), (9000, 100, 5000),
                                            (20000, 384, 19000)])
@pytest.mark.parametrize("level", [1.0, 30.0])
def test_keys_of_minus_infinity(shape, N, pre, first, last, level):
    Hq, Hkv, d = shape
    c = Tree([pre, 50], [N, N], N, Hq, Hkv, d, page=16, seed=pre + first, scores=False)
    c.q[..., 0] = 1.0
    at = ints(c.slots[0], torch.int64)
    c.K[at, :, 0] = -level  # (the other keys' logits: far below 0 too, and still the row's largest)
    clean = c.K.clone()
    c.K[at[first:last], :, 0] = -float("inf")
    c.call()
    torch.cuda.synchronize()
    assert c.status.item() == 0
    keep = np.r_[0:first, last:pre]
    K, V, q = bf16_to_f64(clean[at]), bf16_to_f64(c.V[at]), bf16_to_f64(c.q[0])
    rows = np.r_[keep, pre:pre + N]
    want, move, err = attention(q, K[rows], V[rows], len(keep), c.sees[0], d ** -0.5, False)
    rounding = 2.0 ** -16 if pre + N <= 1024 else 2.0 ** -8
    tol = 2.0 ** -8 * np.abs(want) + (rounding + 2 * err + 2.0 ** -20) * move + 2.0 ** -20
    assert (np.abs(bf16_to_f64(c.out[0]) - want) <= tol).all()
