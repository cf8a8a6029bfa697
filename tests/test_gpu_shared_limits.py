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


def attention_without(c, b, missing):
    """Output and sum of weights times |V| of sequence b's rows in float64, its own rows `missing` left out."""
    from tests.parity import bf16_to_f64
    n, t = c.n[b], c.tok[b]
    G = c.Hq // c.Hkv
    K = np.concatenate([bf16_to_f64(c.K)[t[:n]], bf16_to_f64(c.kn[b])])
    V = np.concatenate([bf16_to_f64(c.V)[t[:n]], bf16_to_f64(c.vn[b])])
    q = bf16_to_f64(c.q[b])
    out, size = np.zeros_like(q), np.zeros_like(q)
    for r in range(c.R):
        use = np.array([i for i in range(n + r + 1) if i - n not in missing])
        for h in range(c.Hq):
            s = K[use, h // G] @ q[r, h] / np.sqrt(c.d)
            w = np.exp(s - s.max())
            w /= w.sum()
            out[r, h], size[r, h] = w @ V[use, h // G], w @ np.abs(V[use, h // G])
    return out, size


@pytest.mark.parametrize("append", [True, False])
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
@pytest.mark.parametrize("private,missing", [([40, 32, 60], [0, 1, 2, 3]), ([40, 30, 60], [2, 3])])
def test_verify_rows_on_a_page_outside_the_pool_are_reported_and_skipped(private, missing, bad, append):
    # sequence 1's rows begin at (or two tokens before) the page after its prefix's, which it does not have, as
    # after a pool that ran out; in the second shape there are enough rows for a combine of eight a CTA
    for others, kw in ((0, dict()), (17, dict(Hq=32, Hkv=8, d=128))):
        c = Case([3, others], [256, 16], [private, list(range(others))], gamma=3, append=append, **kw)
        b, n = 1, c.n[1]
        from tests.parity import bf16_to_f64
        ref, size = attention_without(c, b, missing if not append else [])
        K0, V0 = c.K.clone(), c.V.clone()
        c.table[b, -(-n // 16)] = bad
        c.call()
        c.check(skip=[b], status=vb.VG_ERR_DEVICE_BOUNDS, K0=K0, V0=V0)
        err = np.abs(bf16_to_f64(c.out[b]) - ref)
        assert (err <= 2.0 ** -8 * (size + 2 * np.abs(ref)) + 2.0 ** -14 * size).all(), err.max()
        # what has a place was appended, and nothing else was written
        new = [t[k:] for t, k in zip(c.tok, c.n)]
        new[b] = new[b][:c.R - len(missing)]
        if append:
            assert torch.equal(c.K[torch.from_numpy(new[b]).cuda()], c.kn[b, :c.R - len(missing)])
        rest = np.setdiff1d(np.arange(c.K.shape[0]), np.concatenate(new) if append else [])
        rest = torch.from_numpy(rest).cuda()
        assert torch.equal(c.K[rest].view(torch.int16), K0[rest].view(torch.int16))
        assert torch.equal(c.V[rest].view(torch.int16), V0[rest].view(torch.int16))


# With d = 128 a batch's layout (5 (n_groups + 1) + 4 B + 2 integers) takes the fifth tile's place from about 86
# sequences on: the attention kernel's ring then has four, the fewest that its waits allow.
FOUR_TILES = {
    "two_heads_a_step": dict(members=[128], shared=[1500], private=[[(29 * i) % 400 for i in range(128)]], Hq=4, Hkv=4),
    "one_kv_head": dict(members=[90], shared=[700], private=[[(31 * i) % 300 for i in range(90)]], Hq=1, Hkv=1, gamma=0),
    "odd_kv_heads": dict(members=[60, 40], shared=[900, 128], private=[[(37 * i) % 500 for i in range(60)], [3] * 40],
                         Hq=6, Hkv=3, gamma=2),
    "row_tile_pairs": dict(members=[128], shared=[1300], private=[[(41 * i) % 260 for i in range(128)]], Hq=16, Hkv=4,
                           gamma=3, page=64),
    "many_groups": dict(members=[3] * 40, shared=[128 + 50 * i for i in range(40)], private=[[0, 129, 257]] * 40, Hq=8,
                        Hkv=2, gamma=1),
    "slot_pool": dict(members=[100], shared=[600], private=[[(17 * i) % 300 for i in range(100)]], Hq=8, Hkv=4, page=0),
    "long_private": dict(members=[50, 50], shared=[300, 0], private=[[(97 * i) % 3000 for i in range(50)], [40 * i for i in range(50)]],
                         Hq=8, Hkv=2, gamma=3),
    "largest_batch": dict(members=[1000, 24], shared=[300, 130], private=[[(37 * i) % 150 for i in range(1000)], [5] * 24],
                          Hq=2, Hkv=2),
}


@pytest.mark.parametrize("name", list(FOUR_TILES))
def test_a_ring_of_four_tiles(name):
    kw = dict(d=128, page=16, scores=name != "long_private")
    kw.update(FOUR_TILES[name])
    c = Case(**kw)
    assert 5 * (len(c.members) + 1) + 4 * c.B + 2 > 360
    K0, V0 = c.K.clone(), c.V.clone()
    c.call()
    first = c.out.clone()
    c.check(K0=K0, V0=V0)
    c.K.copy_(K0)
    c.V.copy_(V0)
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int16), c.out.view(torch.int16))
