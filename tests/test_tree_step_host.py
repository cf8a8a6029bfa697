"""What TreeStep refuses, on the CPU: each refusal comes before any call of the library, which a recorder stands in for."""
import pytest

torch = pytest.importorskip("torch")

from self_speculative_sparse_gb300 import binding as vb  # noqa: E402

B, HQ, HKV, D, N, LEN = 2, 8, 2, 64, 70, 100


@pytest.fixture
def calls(monkeypatch):
    seen = []
    monkeypatch.setattr(vb, "vg_tree_verify_workspace_size", lambda dims, n: 256)
    for name in ("vg_tree_build", "vg_rope_append_at", "vg_tree_verify_attn", "vg_sample", "vg_tree_accept"):
        monkeypatch.setattr(vb, name, lambda *a, _name=name, **k: seen.append(_name))
    return seen


def layer(slots=400, heads=HKV, d=D, dtype=torch.bfloat16):
    return torch.zeros((slots, heads, d), dtype=dtype)


def make(layers=None, prefix=None, **where):
    from self_speculative_sparse_gb300.runtime import TreeStep
    where = where or dict(seq_offset=torch.tensor([0, 200]))
    prefix = torch.zeros(B, dtype=torch.int32) if prefix is None else prefix
    return TreeStep(B, HQ, HKV, D, N, LEN, layers or [(layer(), layer())], prefix, **where)


def test_layers_of_other_slots_are_refused(calls):
    make()
    make([(layer().view(400, HKV * D), layer())])
    for K, V in ((layer(d=128), layer(d=128)), (layer(heads=1), layer(heads=1)), (layer(heads=3), layer(heads=3)),
                 (layer(dtype=torch.float32, d=32), layer(dtype=torch.float32, d=32)), (layer(), layer(dtype=torch.float16))):
        with pytest.raises(ValueError, match="layer 0"):
            make([(K, V)])
    with pytest.raises(ValueError, match="layer 1"):
        make([(layer(), layer()), (layer(d=128), layer(d=128))])


def test_where_the_tokens_lie_is_checked(calls):
    table = torch.zeros((B, 12), dtype=torch.int32)
    make(page_table=table, page_size=16)
    make(page_table=torch.zeros((B + 3, 12), dtype=torch.int32), page_size=16)
    for bad in (dict(seq_offset=None), dict(seq_offset=torch.tensor([0, 200]), page_table=table, page_size=16),
                dict(seq_offset=torch.tensor([0])), dict(seq_offset=torch.tensor([0, 200], dtype=torch.int32)),
                dict(seq_offset=torch.tensor([0, 1, 200, 3])[::2]), dict(page_table=table.long(), page_size=16),
                dict(page_table=table[:1], page_size=16), dict(page_table=table.t().contiguous().t(), page_size=16),
                dict(page_table=table[0], page_size=16)):
        with pytest.raises(ValueError):
            make(**bad)
    for bad in (torch.zeros(1, dtype=torch.int32), torch.zeros(B), torch.zeros(B, dtype=torch.int64),
                torch.zeros(2 * B, dtype=torch.int32)[::2], torch.zeros((B, 1), dtype=torch.int32)):
        with pytest.raises(ValueError, match="prefix_len"):
            make(prefix=bad)


def test_scores_and_their_rows_are_checked(calls):
    step = make()
    q = torch.zeros(B * N, HQ, D, dtype=torch.bfloat16)
    out, rows, scores = q.clone(), torch.zeros((B, 2), dtype=torch.int64), torch.zeros((B, LEN))
    step.verify(0, q, out)
    step.verify(0, q, out, rows, scores)
    step.verify(0, q, out, rows, torch.zeros((B, 2 * LEN))[:, :LEN])
    step.verify(0, q, out, rows.view(torch.uint64), scores)
    assert calls == ["vg_tree_verify_attn"] * 4
    for r, s in ((rows, None), (None, scores), (rows.int(), scores), (rows[:, :1], scores), (rows[:1], scores),
                 (torch.zeros((B, 3), dtype=torch.int64), scores), (torch.zeros((2, B), dtype=torch.int64).t(), scores),
                 (rows.view(-1), scores), (rows, scores[:, :-1]), (rows, scores[:1]), (rows, scores.double()),
                 (rows, scores.to(torch.bfloat16)), (rows, torch.zeros((LEN, B)).t()), (rows, scores.view(-1)),
                 (rows, scores.to("meta")), (rows.to("meta"), scores)):
        with pytest.raises(ValueError):
            step.verify(0, q, out, r, s)
    assert len(calls) == 4


def test_what_is_sampled_from_is_checked(calls):
    step = make()
    x, u = torch.zeros((B * N, 50)), torch.zeros(B * N)
    params = vb.make_sampling(torch.ones(B), rows_per_set=N, set_rows=step.len)
    step.sample(x, params, u)
    step.sample(x, params, u.view(B, N))
    assert calls == ["vg_sample"] * 2
    for logits, v in ((x, torch.zeros(2 * B * N)[::2]), (x, torch.zeros((N, B)).t()), (x, u[:-1]), (x, u.double()),
                      (x.to("meta"), u), (x, u.to("meta")), (x.double(), u), (x.t(), u)):
        with pytest.raises(ValueError):
            step.sample(logits, params, v)
    with pytest.raises(ValueError):
        step.sample(x, vb.make_sampling(torch.ones(B, device="meta"), rows_per_set=N), u)
    assert len(calls) == 2
