"""How exact vg_shared_verify_attn is where a row's weight sits on a few keys whose values differ: as exact as
vg_verify_attn, which it stands for.

Bounds, from the arithmetic.  Rows of at most 1024 prefix tokens carry their weights to 2^-17 (a bf16 high and
low part), so what is left is the output's own rounding, half a step: 2^-8 |out|, and 2^-13 A, A = sum_i p_i |v_i|,
for fp32 logits, exponentials and sums: a product of up to 2^10 before its scale of 2^-3 or less, summed in eight
additions each off by 2^-23 of it, moves a logit by less than 2^-14 and a weight by that of it, once in the weights
and once in their sum; the rest is below 2^-17.  Longer rows have weights of one bf16, p_i (1 + e_i) with |e_i| <= 2^-8,
divided by the sum of those same weights: out is off by sum_i p_i e_i (v_i - out), at most
2^-8 sum_i p_i |v_i - out| <= 2^-8 sqrt(sum_i p_i v_i^2 - out^2), before its rounding (to second order, which the
factor 1 + 2^-6 covers).  Short rows also have to be within the framework's bound for attention outputs."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from tests.parity import assert_attn_close, bf16_to_f64  # noqa: E402
from tests.test_gpu_shared import LONG, SMALL, Case  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_speculative_sparse_gb300 import build
    build.build()


LIMIT = 1024  # prefix tokens of a row whose weights are carried in two parts


def check(c, short=True):
    """short: the bounds of rows of at most LIMIT tokens (else those of longer rows for all)."""
    torch.cuda.synchronize()
    assert c.status.item() == 0
    K, V, out = bf16_to_f64(c.K), bf16_to_f64(c.V), bf16_to_f64(c.out)
    q, kn, vn = bf16_to_f64(c.q), bf16_to_f64(c.kn), bf16_to_f64(c.vn)
    scale = c.scale or 1.0 / np.sqrt(c.d)
    for b in range(c.B):
        n, t = c.n[b], c.tok[b]
        k, v = K[t[:n]], V[t[:n]]
        ref = oracle.verify_attention(q[b], k, v, kn[b], vn[b], scale)
        A = oracle.verify_attention(q[b], k, np.abs(v), kn[b], np.abs(vn[b]), scale)
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -13 * A
        if short and n <= LIMIT:
            assert_attn_close(out[b], ref, f"sequence {b}")
        else:
            square = oracle.verify_attention(q[b], k, v * v, kn[b], vn[b] * vn[b], scale)
            tol = tol + (1 + 2.0 ** -6) * 2.0 ** -8 * np.sqrt(np.maximum(square - ref * ref, 0.0))
        err = np.abs(out[b] - ref)
        assert (err <= tol).all(), (b, n, int((err > tol).sum()), (err - tol).max())


def peaked(c, hot, shift=8.0, seed=5):
    """Three keys along one direction, at the places that `hot` gives for each sequence, and every query moved along
    it: nearly all of a row's weight sits on them.  Places inside a shared prefix have to be the members' own too."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    u = torch.randn(c.d, generator=g, device="cuda")
    u *= (c.d / 128) ** 0.5 / u.norm()  # (the logits do not depend on d)
    for b in range(c.B):
        for size, p in zip((50.0, 48.5, 47.0), hot(b)):
            c.K[int(c.tok[b][p])] = (size * u).to(torch.bfloat16)
    c.q += (shift * u / u.norm() ** 2 * (c.d / 128) ** 0.5).to(torch.bfloat16)
    return c


# two or three of them in one tile of 128 keys, so that one run has to weigh them against each other
HOT = {
    "shared": lambda c, s: lambda b: (3, 61, 100),
    "private": lambda c, s: lambda b: (s, s + 40, c.n[b] - 1),
    "both": lambda c, s: lambda b: (5, 77, c.n[b] - 2),
}


@pytest.mark.parametrize("where", list(HOT))
@pytest.mark.parametrize("d", [64, 128])
def test_short_rows_with_weight_on_three_keys(d, where):
    s = 900
    c = Case([12], [s], [[100 + 2 * i for i in range(12)]], Hq=32, Hkv=8, d=d, gamma=7, scores=False, append=False)
    peaked(c, HOT[where](c, s))
    c.call()
    check(c)


@pytest.mark.parametrize("where", list(HOT))
def test_one_token_rows_with_weight_on_three_keys(where):
    s = 900
    c = Case([30, 20], [s, s], [[60 + 2 * i for i in range(30)], [64 + 2 * i for i in range(20)]], Hq=64, Hkv=8, d=128,
             page=64, scores=False)
    peaked(c, HOT[where](c, s))
    c.call()
    check(c)


@pytest.mark.parametrize("n", [1023, 1024, 1025])
def test_rows_at_the_limit(n):
    c = Case([4], [n - 200], [[200] * 4], Hq=16, Hkv=4, d=128, gamma=7, append=False)
    peaked(c, HOT["both"](c, n - 200))
    c.call()
    check(c)


@pytest.mark.parametrize("where", list(HOT))
def test_long_rows_with_weight_on_three_keys(where):
    s = 4096
    c = Case([3], [s], [[100, 700, 1904]], Hq=32, Hkv=8, d=128, gamma=7, append=False)
    peaked(c, HOT[where](c, s))
    c.call()
    check(c)


@pytest.mark.parametrize("where", list(HOT))
def test_short_and_long_rows_of_a_group(where):
    s = 400  # a shared range in two parts, private ranges in two or in one
    c = Case([6], [s], [[50, 300, 624, 625, 1500, 4000]], Hq=32, Hkv=8, d=128, gamma=7, append=False)
    peaked(c, HOT[where](c, s))
    c.call()
    check(c)


@pytest.mark.parametrize("name", [*SMALL, *LONG])
def test_the_weights_of_the_shared_tests_cases(name):
    c = Case(**{**SMALL, **LONG}[name])
    K0, V0 = c.K.clone(), c.V.clone()
    c.call()
    c.K, c.V = K0, V0
    check(c)


@pytest.mark.parametrize("shared,private", [(900, [100, 60, 0]), (4000, [300, 0, 2000]), (100, [3000, 500, 1000])])
def test_weights_sum_to_one(shared, private):
    # with equal values of all tokens a row's output is that value, whatever its weights: their sum is off by
    # fp32 roundings only, far less than half a step of the output
    c = Case([3], [shared], [private], Hq=32, Hkv=8, d=128, gamma=7, append=False)
    peaked(c, lambda b: (3, 61, shared - 1))
    c.V.fill_(1.5)
    c.vn.fill_(1.5)
    c.call()
    torch.cuda.synchronize()
    assert c.status.item() == 0 and (c.out == 1.5).all(), (c.out != 1.5).sum().item()
