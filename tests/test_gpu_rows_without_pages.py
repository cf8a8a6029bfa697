"""Rows of a block table that were not grown for the tokens a call is about to write (a page pool that ran out
leaves such rows): vg_verify_attn and vg_sparse_draft_attn report the tokens that have no place, give their keys no
weight when they would come from the cache, and serve every other sequence."""
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


@pytest.mark.parametrize("bad", [-1, 10 ** 6])
@pytest.mark.parametrize("k", [8, 200])  # a sequence's entries in one CTA (finished there), and in several
def test_a_draft_token_without_a_place(k, bad):
    c = Case([3], [0], [[300, 320, 301]], scores=False)  # sequence 1's token 320 begins a page
    b, g = 1, torch.Generator(device="cuda").manual_seed(1)
    idx = torch.stack([torch.randperm(300, generator=g, device="cuda")[:k].sort().values for _ in range(3)]).to(torch.int32)
    count = torch.full((3,), k, dtype=torch.int32, device="cuda")
    tail = torch.ones(3, dtype=torch.int32, device="cuda")
    q, kn, vn = c.q[:, 0], c.kn[:, 0].contiguous(), c.vn[:, 0].contiguous()
    out = torch.full((3, c.Hq, c.d), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(vb.vg_workspace_size(c.dims, k), dtype=torch.uint8, device="cuda")
    K0, V0 = c.K.clone(), c.V.clone()
    c.table[b, 320 // 16] = bad
    vb.vg_sparse_draft_attn(c.dims, c.cache, q.contiguous(), kn, vn, idx, count, k, c.prefix, tail, out, ws,
                            dev_status=c.status)
    torch.cuda.synchronize()
    assert c.status.item() == vb.VG_ERR_DEVICE_BOUNDS
    for i in range(3):  # (the token itself comes from the inputs)
        t, n = c.tok[i], c.n[i]
        ref = oracle.draft_step(bf16_to_f64(q[i]), bf16_to_f64(K0)[t[:n]], bf16_to_f64(V0)[t[:n]], idx[i].cpu().numpy(),
                                bf16_to_f64(kn[i:i + 1]), bf16_to_f64(vn[i:i + 1]))
        assert_attn_close(bf16_to_f64(out[i]), ref, f"sequence {i}")
    new = [c.tok[i][c.n[i]] for i in (0, 2)]
    for i, s in zip((0, 2), new):
        assert torch.equal(c.K[int(s)], kn[i]) and torch.equal(c.V[int(s)], vn[i])
    rest = torch.from_numpy(np.setdiff1d(np.arange(c.K.shape[0]), new)).cuda()
    assert torch.equal(c.K[rest].view(torch.int16), K0[rest].view(torch.int16))
    assert torch.equal(c.V[rest].view(torch.int16), V0[rest].view(torch.int16))
