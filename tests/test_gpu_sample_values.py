"""What vg_sample returns beside the token, at the edges of its parameters: probabilities and filtered logits.

A probability is a weight over the sum of n, each off by at most 2^-28 of itself and 2^-40 of the largest, rounded once: 2^-24
(half a step of fp32) and 2^-27 of its value p, 2^-50 for what is of second order, and 2^-40 (1 + n p) of the largest probability.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_sample import Rows, fast_row, logits  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_speculative_sparse_gb300 import build
    build.build()


# (every end of a row: few candidates, up to 2048 of them, each CTA's own, and a pass over the row)
@pytest.mark.parametrize("V,par", [(50, dict()), (3000, dict(k=40)), (30000, dict(k=1500)), (30000, dict(k=9000)),
                                   (30000, dict(p=0.9)), (30000, dict()), (30000, dict(T=3.0, p=0.97))])
def test_a_probability_is_rounded_once(V, par):
    c = Rows(logits(64, V, spread=1.5, seed=V), seed=V + 1, **par).call(filtered=False)
    T, k, p, m = (float(t[0]) for t in (c.T, c.k, c.p, c.m))
    for r in range(c.n):
        token, want, kept = fast_row(c.ref[r], float(c.u[r]), T, int(k), p, m)
        x = c.ref[r][kept].astype(np.float64)
        most = 1 / np.exp((x - x.max()) / T).sum()
        assert c.token[r].item() == token
        tol = want * (2.0 ** -24 + 2.0 ** -27 + 2.0 ** -50) + 2.0 ** -40 * (1 + len(kept) * want) * most
        assert abs(c.prob[r].item() - want) <= tol
