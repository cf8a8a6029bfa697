"""vg_accept on logits far from zero, as vg_sample's filtered rows of a low temperature are.

A softmax does not change when a row's logits are shifted: logits of whole eighths, shifted by numbers that keep them exact
in fp32, give the decisions of the rows as they were (inputs as in test_gpu_accept.py, clear of every boundary).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from self_speculative_sparse_gb300 import binding as vb  # noqa: E402
from tests.test_gpu_accept import _clear_of_boundaries, _run  # noqa: E402
from tests.test_gpu_sample import Rows, logits  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_speculative_sparse_gb300 import build
    build.build()


@pytest.mark.parametrize("mode", ["sample", "greedy"])
@pytest.mark.parametrize("V", [50, 1001, 40000])
@pytest.mark.parametrize("shift", [2.0 ** 17, -2.0 ** 17, 2.0 ** 20, -2.0 ** 20])
def test_shifted_rows(shift, V, mode):
    r = np.random.default_rng(V)
    B, gamma = 6, 4
    p = np.round(r.normal(size=(B, gamma + 1, V)) * 16) / 8
    q = p[:, :gamma] + np.round(r.normal(size=(B, gamma, V)) * 4) / 8
    x = np.array([[r.choice(V, p=oracle.softmax(q[b, t])) for t in range(gamma)] for b in range(B)], dtype=np.int32)
    if mode == "greedy":
        x[:3] = p[:3, :gamma].argmax(-1)
    inp = dict(p_logits=p.astype(np.float32), q_logits=q.astype(np.float32), x=x, u=r.random((B, gamma), dtype=np.float32),
               u_res=r.random(B, dtype=np.float32))
    _clear_of_boundaries(inp, r)
    want = _run(inp, mode)
    far = dict(inp, p_logits=(p + shift).astype(np.float32), q_logits=(q - shift).astype(np.float32))
    assert np.array_equal(far["p_logits"].astype(np.float64) - shift, p)
    got = _run(far, mode)
    for a, b in zip(want[:2], got[:2]):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 32, 2.0 ** 60, 2.0 ** 100])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_rows_that_are_one_token(size, sign):
    """Logits this far apart leave all weight on the largest: p is accepted where the draft names it, whatever q is."""
    r = np.random.default_rng(3)
    B, gamma, V = 5, 3, 9000
    p = (np.stack([[r.permutation(V) for _ in range(gamma + 1)] for _ in range(B)]) + (1.0 if sign > 0 else -V)) * size
    best = p.argmax(-1).astype(np.int32)
    x = best[:, :gamma].copy()
    for b in range(1, B):
        if b <= gamma:
            x[b, b - 1] = (x[b, b - 1] + 1) % V
    inp = dict(p_logits=p.astype(np.float32), q_logits=np.zeros((B, gamma, V), np.float32), x=x,
               u=np.full((B, gamma), 0.5, np.float32), u_res=np.full(B, 0.5, np.float32))
    for mode in ("sample", "greedy"):
        n, nxt = _run(inp, mode)[:2]
        assert n.tolist() == [gamma, 0, 1, 2, gamma]
        assert nxt.tolist() == [best[b, a] for b, a in enumerate(n)]


def test_rows_at_a_tiny_temperature_serve_the_acceptance():
    """A distribution that is one token, of negative logits: the chain's acceptance keeps exactly that token."""
    V = 500
    x = logits(8, V, seed=4) - 40
    c = Rows(x, T=1e-38).call()
    best = x.argmax(1)
    assert c.token.tolist() == best.tolist() and (c.prob == 1).all()
    p = c.filtered[:, :V].contiguous().view(4, 2, V)
    draft = torch.tensor(best.reshape(4, 2)[:, :1].astype(np.int32).copy(), device="cuda")
    draft[3] = (draft[3] + 1) % V
    ws = torch.empty(vb.vg_accept_workspace_size(4, 1, V), dtype=torch.uint8, device="cuda")
    n, nxt = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    q = torch.zeros(4, 1, V, device="cuda")
    vb.vg_accept(4, 1, V, p, q, draft, torch.full((4, 1), 0.5, device="cuda"), torch.full((4,), 0.5, device="cuda"),
                 vb.VG_ACCEPT_SAMPLE, n, nxt, None, ws)
    assert n.tolist() == [1, 1, 1, 0] and nxt.tolist() == best.reshape(4, 2)[[0, 1, 2, 3], [1, 1, 1, 0]].tolist()
