"""vg_tree_verify_attn with a sequence out of range: it is reported, and neither its outputs nor its scores nor the cache
are touched, whatever the workspace holds; the others are served (against attention in float64, as in their own test)."""
import pytest

torch = pytest.importorskip("torch")

from self_speculative_sparse_gb300 import binding as vb  # noqa: E402
from tests.test_gpu_tree_attn import Tree, ints  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_speculative_sparse_gb300 import build
    build.build()


def left_alone(c, b, lens):
    """The call with these node counts leaves sequence b's outputs and scores alone, and the cache but for the others' nodes."""
    c.tree = vb.make_tree(c.N, c.visible, ints(lens))
    c.ws.view(torch.float32).fill_(7.0)
    K, V = c.K.clone(), c.V.clone()
    c.call()
    torch.cuda.synchronize()
    assert c.status.item() == vb.VG_ERR_DEVICE_BOUNDS
    assert (c.out[b] == 9).all()
    if c.scores is not None:
        assert (c.scores[b] == 9).all()
    mine = torch.ones(c.K.shape[0], dtype=torch.bool, device="cuda")
    if c.fresh:
        for x in range(c.B):
            if x != b:
                mine[ints(c.slots[x][c.pre[x]:], torch.int64)] = False
    for new, old in ((c.K, K), (c.V, V)):
        assert torch.equal(new[mine].view(torch.int16), old[mine].view(torch.int16))
    c.lens[b] = 0
    c.check(skip=(b,))


@pytest.mark.parametrize("fresh", [True, False])
@pytest.mark.parametrize("scores", [True, False])
def test_a_slot_pool_that_ends_before_the_nodes(fresh, scores):
    c = Tree([300, 20], [27, 9], 27, page=0, seed=9, fresh=fresh, scores=scores, tight=True)
    assert int(c.off[1]) + 20 + 27 > c.K.shape[0] >= int(c.off[1]) + 20
    left_alone(c, 1, [27, 27])


@pytest.mark.parametrize("fresh", [True, False])
@pytest.mark.parametrize("scores", [True, False])
@pytest.mark.parametrize("page", [8, 16, 64])
def test_a_table_row_too_short_for_the_nodes(fresh, scores, page):
    N = 90
    c = Tree([640 - 27, 20, 100], [27, 9, 0], N, page=page, seed=5, fresh=fresh, scores=scores)
    assert c.table.shape[1] * page == 640
    left_alone(c, 0, [28, 9, 0])


@pytest.mark.parametrize("offset", [-1, -(1 << 40), 1 << 20, (1 << 62)])
def test_a_sequence_that_begins_outside_the_pool(offset):
    c = Tree([300, 20, 70], [27, 9, 27], 27, page=0, seed=3, fresh=True)
    c.off[1] = offset
    left_alone(c, 1, [27, 9, 27])


@pytest.mark.parametrize("fresh", [True, False])
@pytest.mark.parametrize("pre,nodes", [(501, 27), (-1, 27), (500, 28), (500, -1)])
def test_lengths_out_of_range(pre, nodes, fresh):
    c = Tree([300, 20, 500, 7], [27, 3, 27, 27], 27, seed=9, fresh=fresh, max_len=500)
    c.prefix[2] = pre
    left_alone(c, 2, [27, 3, nodes, 27])
