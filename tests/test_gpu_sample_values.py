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


MOST = float(np.finfo(np.float32).max)


def filtered(c, r, kept):
    """The definition: a kept logit over T (taken to lie in [2^-70, 2^70]), one rounding, held within the finite floats."""
    t = np.float32(min(max(float(c.T[r]), 2.0 ** -70), 2.0 ** 70))
    ref = np.full(c.V, -np.inf, np.float32)
    with np.errstate(over="ignore"):
        ref[kept] = np.clip(np.minimum(c.ref[r][kept], np.float32(MOST)) / t, -MOST, MOST)
    return ref, float(t)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [50, 30000])
@pytest.mark.parametrize("T,size,shift", [
    (1e-38, 3.0, -40.0), (1e-38, 3.0, 40.0), (1e-38, 1e-21, 0.0), (1e-38, 1e-21, -1e-20), (1.4e-45, 1.0, 0.0), (1e-20, 1e-20, 0.0),
    (1e-10, 1e33, 0.0), (0.25, 3e37, -3e38), (1e-3, 1e37, 0.0), (2.0 ** 65, 2e19, 0.0), (3e38, 1.0, 0.0), (1e25, 1e21, 0.0)])
@pytest.mark.parametrize("par", [dict(), dict(p=0.8), dict(k=5)])
def test_filtered_logits_are_finite_at_every_temperature(T, size, shift, V, dtype, par):
    x = np.clip(logits(3, V, spread=1.0, seed=7) * size + shift, -MOST / 2, MOST / 2)
    c = Rows(x, T=T, dtype=dtype, seed=2, **par).call()
    assert c.status.item() == 0
    k, p = par.get("k", 0), float(np.float32(par.get("p", 1.0)))
    for r in range(c.n):
        token, _, kept = fast_row(c.ref[r], float(c.u[r]), filtered(c, r, [])[1], k, p, 0.0)
        got = c.filtered[r, :V].cpu().numpy()
        assert np.array_equal(got, filtered(c, r, kept)[0])
        assert np.isfinite(got[kept]).all()
        assert c.token[r].item() == token


@pytest.mark.parametrize("m", [0.0, -0.0, -1e-45, -0.5, -float("inf")])
@pytest.mark.parametrize("V,par", [(300, dict()), (30000, dict(p=0.9)), (30000, dict(k=40))])
def test_a_min_p_of_0_or_less_is_off(m, V, par):
    x = logits(3, V, seed=5)
    on, off = Rows(x, m=m, **par).call(), Rows(x, **par).call()
    off.params.min_p = None
    off.call()
    assert on.status.item() == 0
    for a, b in ((on.token, off.token), (on.prob, off.prob), (on.filtered, off.filtered)):
        assert torch.equal(a, b)
