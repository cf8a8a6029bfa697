"""vg_shared_verify_attn where its inputs are out of range: what is reported, what is still served, and
that nothing outside the outputs is touched.  Tolerances are those of the shared verification's own test."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from self_speculative_sparse_gb300 import binding as vb  # noqa: E402
from tests.test_gpu_shared import Case  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_speculative_sparse_gb300 import build
    build.build()


GUARD = 4096  # floats before and behind the score rows


def guarded_scores(c):
    """Puts the case's score rows between guards; the whole buffer."""
    whole = torch.full((c.B * c.stride + 2 * GUARD,), 7.0, device="cuda")
    c.scores = whole[GUARD:GUARD + c.B * c.stride].view(c.B, c.stride)
    return whole


def guards_hold(whole):
    return bool((whole[:GUARD] == 7.0).all()) and bool((whole[-GUARD:] == 7.0).all())


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("bad_first_length", [False, True])
@pytest.mark.parametrize("group", [0, 1])
@pytest.mark.parametrize("value", [-1, -127, -128, -129, -500, -4096, -(1 << 31)])
def test_a_negative_shared_length_is_reported_and_the_group_read_by_itself(value, group, bad_first_length, page):
    c = Case([2, 3], [300, 513], [[5, 0], [1, 130, 2]], gamma=3, page=page)
    whole = guarded_scores(c)
    K0, V0 = c.K.clone(), c.V.clone()
    c.shared_len[group] = value
    skip = []
    if bad_first_length:  # of the same group: there is then no row to read a prefix through either
        skip = [2 * group]
        c.prefix[skip[0]] = -1
    c.call()
    c.check(skip=skip, status=vb.VG_ERR_DEVICE_BOUNDS, K0=K0, V0=V0)
    assert guards_hold(whole)
    for b in skip:
        assert torch.isnan(c.out[b]).all() and (c.scores[b] == 7.0).all()


@pytest.mark.parametrize("value", [514, 1 << 20, (1 << 31) - 1])
def test_a_shared_length_beyond_a_member_is_reported_and_the_group_read_by_itself(value):
    c = Case([2, 3], [300, 513], [[5, 0], [1, 0, 2]], gamma=1)
    whole = guarded_scores(c)
    K0, V0 = c.K.clone(), c.V.clone()
    c.shared_len[1] = value
    c.call()
    c.check(status=vb.VG_ERR_DEVICE_BOUNDS, K0=K0, V0=V0)
    assert guards_hold(whole)
