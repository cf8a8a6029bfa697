"""Rows of a block table that were not grown for the tokens a call is about to write (a page pool that ran out
leaves such rows): vg_verify_attn reports the verify rows that have no place, gives their keys no weight when
they would come from the cache, and serves every other sequence."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from self_speculative_sparse_gb300 import binding as vb  # noqa: E402
from tests.parity import assert_attn_close, bf16_to_f64  # noqa: E402
from tests.test_gpu_shared import Case  # noqa: E402
from tests.test_gpu_shared_limits import attention_without  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_speculative_sparse_gb300 import build
    build.build()


def verify(c):
    ws = torch.empty(vb.vg_workspace_size(c.dims, 16), dtype=torch.uint8, device="cuda")
    vb.vg_verify_attn(c.dims, c.cache, c.q, c.kn if c.append else None, c.vn if c.append else None, c.prefix, c.mask, 0,
                      c.scores, None, c.stride, c.out, ws, dev_status=c.status)
    torch.cuda.synchronize()


@pytest.mark.parametrize("append", [True, False])
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
@pytest.mark.parametrize("private,missing", [([40, 32, 60], [0, 1, 2, 3]), ([40, 30, 60], [2, 3])])
@pytest.mark.parametrize("others,kw", [(0, dict()), (21, dict(Hq=32, Hkv=8, d=128))])  # a narrow and a wide combine
def test_verify_rows_without_a_place(others, kw, private, missing, bad, append):
    c = Case([3, others], [256, 16], [private, list(range(others))], gamma=3, append=append, **kw)
    b, n = 1, c.n[1]
    ref, _ = attention_without(c, b, missing if not append else [])
    want = [oracle.verify_attention(bf16_to_f64(c.q[i]), *(bf16_to_f64(x)[c.tok[i][:c.n[i]]] for x in (c.K, c.V)),
                                    bf16_to_f64(c.kn[i]), bf16_to_f64(c.vn[i])) for i in range(c.B)]
    want[b] = ref
    K0, V0 = c.K.clone(), c.V.clone()
    c.table[b, -(-n // 16)] = bad
    verify(c)
    assert c.status.item() == vb.VG_ERR_DEVICE_BOUNDS
    for i in range(c.B):
        assert_attn_close(bf16_to_f64(c.out[i]), want[i], f"sequence {i}")
    new = [t[k:] for t, k in zip(c.tok, c.n)]
    new[b] = new[b][:c.R - len(missing)]
    if append:
        for i in range(c.B):
            at = torch.from_numpy(new[i]).cuda()
            assert torch.equal(c.K[at], c.kn[i, :len(new[i])]) and torch.equal(c.V[at], c.vn[i, :len(new[i])])
    rest = torch.from_numpy(np.setdiff1d(np.arange(c.K.shape[0]), np.concatenate(new) if append else [])).cuda()
    assert torch.equal(c.K[rest].view(torch.int16), K0[rest].view(torch.int16))
    assert torch.equal(c.V[rest].view(torch.int16), V0[rest].view(torch.int16))


@pytest.mark.parametrize("append", [True, False])
def test_rows_that_all_have_a_place_report_nothing(append):
    for others, kw in ((0, dict()), (21, dict(Hq=32, Hkv=8, d=128))):
        c = Case([3, others], [256, 16], [[40, 30, 60], list(range(others))], gamma=3, append=append, **kw)
        verify(c)
        assert c.status.item() == 0
