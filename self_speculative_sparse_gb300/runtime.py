"""Device-resident state of one Vegas layer and the calls that run on it.

``LayerState`` owns the torch tensors the C ABI works on: the token-granular KV
slot pool, per-sequence offsets and lengths, the iteration's inputs, output
buffers, the workspace and the device status word.  ``PagePool`` owns the block table,
page counts and references that the layers of a paged cache share, ``TreeStep`` what a step with a
tree of drafted tokens needs.  Their methods only
marshal arguments to libvg.so (via ``binding``); PyTorch serves as the allocator and the
stream provider.
"""
from __future__ import annotations

import numpy as np
import torch

from . import binding as vb


def bf16_tensor(a: np.ndarray, device) -> torch.Tensor:
    """bf16 bit patterns (numpy uint16) -> a torch.bfloat16 tensor on `device`."""
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).to(device).view(torch.bfloat16)


def bf16_bits(t: torch.Tensor) -> np.ndarray:
    """torch.bfloat16 tensor -> numpy uint16 bit patterns (host copy)."""
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


class LayerState:
    """One layer's cache, inputs and outputs on the GPU.

    pool: the dict produced by ``Workload.layer_pool`` (host arrays)."""

    def __init__(self, w, pool: dict, device="cuda", k: int | None = None, mask0: int | None = None,
                 mask1: int | None = None, max_len: int | None = None):
        self.w = w
        self.device = torch.device(device)
        dev = self.device
        self.B, self.Hq, self.Hkv, self.d, self.gamma = w.B, w.Hq, w.Hkv, w.d, w.gamma
        self.k = w.k if k is None else k
        self.max_len = int(pool["prefix_len"].max()) if max_len is None else max_len
        self.mask0 = w.row_mask(w.select_rows) if mask0 is None else mask0
        self.mask1 = w.row_mask(w.extra_rows) if mask1 is None else mask1
        self.K = bf16_tensor(pool["K"], dev)
        self.V = bf16_tensor(pool["V"], dev)
        self.seq_offset = torch.from_numpy(pool["seq_offset"].astype(np.int64)).to(dev)
        self.prefix_len = torch.from_numpy(pool["prefix_len"].astype(np.int32)).to(dev)
        self.q_verify = bf16_tensor(pool["q_verify"], dev)
        self.k_new = bf16_tensor(pool["k_new"], dev)
        self.v_new = bf16_tensor(pool["v_new"], dev)
        self.q_draft = bf16_tensor(pool["q_draft"], dev)
        self.k_draft = bf16_tensor(pool["k_draft"], dev)
        self.v_draft = bf16_tensor(pool["v_draft"], dev)
        self.dims = vb.make_dims(self.B, self.Hq, self.Hkv, self.d, self.gamma, self.max_len)
        if "page_table" in pool:  # a paged layout of the same layer (seq_offset then unused)
            self.page_table = torch.from_numpy(pool["page_table"].astype(np.int32)).to(dev)
            self.cache = vb.make_cache(self.K, self.V, None, page_table=self.page_table,
                                       page_size=int(pool["page_size"]))
        else:
            self.page_table = None
            self.cache = vb.make_cache(self.K, self.V, self.seq_offset)
        R = self.gamma + 1
        self.score_stride = max(4, (self.max_len + 3) // 4 * 4)
        self.out_verify = torch.empty(self.B, R, self.Hq, self.d, dtype=torch.bfloat16, device=dev)
        self.scores0 = torch.zeros(self.B, self.score_stride, dtype=torch.float32, device=dev)
        self.scores1 = (torch.zeros(self.B, self.score_stride, dtype=torch.float32, device=dev)
                        if self.mask1 else None)
        self.idx = torch.empty(self.B, self.k, dtype=torch.int32, device=dev)
        self.count = torch.empty(self.B, dtype=torch.int32, device=dev)
        self.idx1 = torch.empty(self.B, self.k, dtype=torch.int32, device=dev) if self.mask1 else None
        self.count1 = torch.empty(self.B, dtype=torch.int32, device=dev) if self.mask1 else None
        self.out_draft = torch.empty(max(self.gamma, 1), self.B, self.Hq, self.d, dtype=torch.bfloat16, device=dev)
        self.ws_bytes = vb.vg_workspace_size(self.dims, self.k)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    # --------------------------------------------------------------- calls
    def _iter_args(self, select_extra: bool):
        ins = vb.vg_iter_inputs(vb.ptr(self.q_verify), vb.ptr(self.k_new), vb.ptr(self.v_new), vb.ptr(self.q_draft),
                                vb.ptr(self.k_draft), vb.ptr(self.v_draft), vb.ptr(self.prefix_len))
        outs = vb.vg_iter_outputs(vb.ptr(self.out_verify), vb.ptr(self.scores0), vb.ptr(self.scores1),
                                  self.score_stride, vb.ptr(self.idx), vb.ptr(self.count),
                                  vb.ptr(self.idx1) if select_extra else None,
                                  vb.ptr(self.count1) if select_extra else None, vb.ptr(self.out_draft))
        return ins, outs

    def iteration(self, stream=None, select_extra: bool = True) -> None:
        """verify -> select -> gamma draft steps, one C call."""
        ins, outs = self._iter_args(select_extra)
        vb.vg_iteration(self.dims, self.cache, ins, self.k, self.mask0, self.mask1, outs, self.ws,
                        dev_status=self.status, stream=stream)

    def plan(self, select_extra: bool = True) -> "IterationPlan":
        """The iteration on this state's current buffers, captured once (vg_iteration_plan_*)."""
        ins, outs = self._iter_args(select_extra)
        h = vb.vg_iteration_plan_create(self.dims, self.cache, ins, self.k, self.mask0, self.mask1, outs, self.ws,
                                        dev_status=self.status)
        return IterationPlan(h, [v for v in vars(self).values() if isinstance(v, torch.Tensor)])

    def verify(self, stream=None, append: bool = True) -> None:
        vb.vg_verify_attn(self.dims, self.cache, self.q_verify, self.k_new if append else None,
                          self.v_new if append else None, self.prefix_len, self.mask0, self.mask1, self.scores0,
                          self.scores1, self.score_stride, self.out_verify, self.ws, dev_status=self.status,
                          stream=stream)

    def select(self, stream=None, which: int = 0) -> None:
        sc, idx, cnt = (self.scores0, self.idx, self.count) if which == 0 else (self.scores1, self.idx1, self.count1)
        vb.vg_topk_select(sc, self.score_stride, self.prefix_len, self.B, self.max_len, self.k, idx, cnt,
                          dev_status=self.status, stream=stream)

    def draft_step(self, s: int, tail_len: torch.Tensor, stream=None, settled: bool | None = None) -> None:
        """Draft step s: attend idx U [n_b, n_b + s], appending draft token s at n_b + s.

        settled (default: s > 0): the selection was made, and the block table last changed, before
        the kernel preceding this call, as it is for every step of a draft phase after the first."""
        settled = s > 0 if settled is None else settled
        vb.vg_sparse_draft_attn(self.dims, self.cache, self.q_draft[s], self.k_draft[s], self.v_draft[s], self.idx,
                                self.count, self.k, self.prefix_len, tail_len, self.out_draft[s], self.ws,
                                dev_status=self.status, stream=stream,
                                flags=vb.VG_DRAFT_SELECTION_SETTLED if settled else 0)

    def verify_shared(self, groups: vb.vg_prefix_groups, ws: torch.Tensor, stream=None, append: bool = True) -> None:
        """``verify`` for groups that share a prefix (vb.make_groups); ws: scratch of
        vb.vg_shared_verify_workspace_size(self.dims, groups) bytes.  Fills out_verify and scores0: a
        state with a second mask, whose scores1 would stay those of an earlier call, is refused."""
        if self.mask1:
            raise ValueError("verify_shared sums the rows of one mask: make the state without a second one")
        vb.vg_shared_verify_attn(self.dims, self.cache, groups, self.q_verify, self.k_new if append else None,
                                 self.v_new if append else None, self.prefix_len, self.mask0, self.scores0,
                                 self.score_stride, self.out_verify, ws, dev_status=self.status, stream=stream)

    def rope_append(self, rope: vb.vg_rope, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                    q_out: torch.Tensor | None = None, stream=None) -> None:
        """Rotate the verify rows' q ([B * (gamma + 1)][H_q][d], in place without q_out) and k, and
        append k and v behind the prefixes (then ``verify(append=False)``)."""
        q_out = q if q_out is None else q_out
        rows = self.B * (self.gamma + 1)
        for name, t, heads in (("q", q, self.Hq), ("k", k, self.Hkv), ("v", v, self.Hkv), ("q_out", q_out, self.Hq)):
            if t.dim() < 2 or t.shape[0] != rows or t[0].numel() != heads * self.d:
                raise ValueError(f"{name}: {rows} rows of {heads} heads of {self.d}, not {tuple(t.shape)}")
            if t.dtype != torch.bfloat16 or t.device != self.K.device:
                raise ValueError(f"{name}: bfloat16 on {self.K.device}, not {t.dtype} on {t.device}")
            if not t[0].is_contiguous():  # (only the rows may be apart)
                raise ValueError(f"{name}: each row's heads must lie together")
        vb.vg_rope_append(self.dims, self.cache, rope, q, q.stride(0), k, k.stride(0), v, v.stride(0), None,
                          rows, self.prefix_len, q_out, q_out.stride(0), dev_status=self.status, stream=stream)

    def launches_per_iteration(self, select_extra: bool = False, tail_from_device: bool = False) -> int:
        """Kernels one iteration enqueues: the verify kernel and its combine, one selection
        (two with select_extra), and each draft step's kernels (vg_iteration gives step s a
        host-known tail of s + 1; the per-step calls here pass a device tail array)."""
        draft = sum(vb.vg_sparse_draft_launches(self.dims, self.k, 0 if tail_from_device else s + 1)
                    for s in range(self.gamma))
        return 2 + (2 if select_extra and self.mask1 else 1) + draft

    def check_status(self) -> int:
        return int(self.status.item())


class PagePool:
    """The pages of a paged cache and the rows that hold them (vg_pages_*), on the device.

    layers: (K, V) tensors [n_pages * page_size][H_kv][d] of each layer; one table serves all."""

    def __init__(self, n_seqs: int, pages_per_seq: int, n_pages: int, page_size: int, layers):
        self.layers = list(layers)
        K = self.layers[0][0]
        dev = K.device
        self.page_size = page_size
        self.token_bytes = K[0].numel() * K.element_size()
        self.page_table = torch.full((n_seqs, pages_per_seq), -1, dtype=torch.int32, device=dev)
        self.held = torch.zeros(n_seqs, dtype=torch.int32, device=dev)
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device=dev)
        self.n_live = torch.zeros(1, dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.pool = vb.make_pages(self.page_table, self.held, self.refs, page_size)
        self.caches = vb.make_caches(self.layers)
        self.ws = torch.empty(vb.vg_pages_workspace_size(self.pool), dtype=torch.uint8, device=dev)

    def cache(self, layer: int = 0) -> vb.vg_kv_cache:
        """Layer `layer` as a paged cache whose sequences are the table's first rows."""
        K, V = self.layers[layer]
        return vb.make_cache(K, V, None, page_table=self.page_table, page_size=self.page_size)

    def _rows(self, **lists) -> int:
        """How many rows a request's lists name, after checking that the kernels can read them."""
        n = lists["length"].numel()
        for name, t in lists.items():
            if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or t.device != self.refs.device:
                raise ValueError(f"{name}: int32 in one dense dimension on {self.refs.device}, not {t.dtype} "
                                 f"{tuple(t.shape)} with strides {t.stride()} on {t.device}")
            if t.numel() != n:
                raise ValueError(f"{name} has {t.numel()} entries, length {n}")
        return n

    def resize(self, seq: torch.Tensor | None, length: torch.Tensor, stream=None) -> None:
        """Rows seq (None: the first ones) hold length tokens each; 0 frees a row.  int32 tensors."""
        n = self._rows(length=length) if seq is None else self._rows(seq=seq, length=length)
        vb.vg_pages_resize(self.pool, seq, length, n, self.ws, dev_status=self.status, stream=stream)

    def fork(self, parent: torch.Tensor, child: torch.Tensor, length: torch.Tensor, room: int = 0,
             stream=None) -> None:
        """Rows child become branches of the first length tokens of rows parent.  int32 tensors."""
        n = self._rows(parent=parent, child=child, length=length)
        vb.vg_pages_fork(self.pool, self.caches, self.token_bytes, parent, child, length, n, room,
                         self.ws, dev_status=self.status, stream=stream)

    def compact(self, stream=None) -> None:
        """Move the live pages to the front of the pool, in place (n_live: how many)."""
        vb.vg_pages_compact(self.pool, self.caches, self.token_bytes, self.page_table, self.refs, self.n_live,
                            self.ws, dev_status=self.status, stream=stream)

    def check_status(self) -> int:
        return int(self.status.item())


class TreeStep:
    """A speculation step with a tree of drafted tokens, over all layers of one cache (vg_tree_*,
    vg_rope_append_at, vg_sample).  Put the drafts into ``parent``, ``len`` and ``tokens``, then call
    build, and for each layer rope_append and verify, then sample on the nodes' logits, then accept.

    layers: (K, V) tensors [slots][H_kv][d] of each layer, located by seq_offset, or by page_table
    with page_size; one table serves all.  prefix_len (int32 [B]) is advanced by accept."""

    def __init__(self, B: int, H_q: int, H_kv: int, d: int, n_nodes: int, max_len: int, layers, prefix_len: torch.Tensor,
                 seq_offset: torch.Tensor | None = None, page_table: torch.Tensor | None = None, page_size: int = 0):
        self.layers = list(layers)
        dev = self.layers[0][0].device
        self.B, self.Hq, self.Hkv, self.d, self.n_nodes = B, H_q, H_kv, d, n_nodes
        self.max_len, self.words = max_len, -(-n_nodes // 64)
        for i, kv in enumerate(self.layers):
            for name, t in zip("KV", kv):
                if t.dtype != torch.bfloat16 or t.shape[1:].numel() != H_kv * d:
                    raise ValueError(f"layer {i}: {name} is {t.dtype} {tuple(t.shape)}: slots of {H_kv} heads of {d} bfloat16")
        if (seq_offset is None) == (page_table is None):
            raise ValueError("seq_offset or page_table")
        self._dense("prefix_len", prefix_len, torch.int32, (B,), dev)
        if page_table is None:
            self._dense("seq_offset", seq_offset, torch.int64, (B,), dev)
        else:
            self._dense("page_table", page_table, torch.int32, (B, 1), dev)
        self.dims = vb.make_dims(B, H_q, H_kv, d, 0, max_len)
        self.cache = [vb.make_cache(K, V, seq_offset, page_table=page_table, page_size=page_size) for K, V in self.layers]
        self.caches = vb.make_caches(self.layers)
        self.prefix_len = prefix_len
        i32 = dict(dtype=torch.int32, device=dev)
        self.parent = torch.full((B, n_nodes), -1, **i32)
        self.len = torch.zeros(B, **i32)
        self.tokens = torch.zeros((B, n_nodes), **i32)
        self.target = torch.zeros((B, n_nodes), **i32)
        self.prob = torch.zeros((B, n_nodes), dtype=torch.float32, device=dev)
        self.visible = torch.zeros((B, n_nodes, self.words), dtype=torch.int64, device=dev)
        self.position = torch.zeros((1, B * n_nodes), **i32)
        self.path = torch.zeros((B, n_nodes), **i32)
        self.n_accept, self.next_token = torch.zeros(B, **i32), torch.zeros(B, **i32)
        self.status = torch.zeros(1, **i32)
        self.tree = vb.make_tree(n_nodes, self.visible, self.len)
        self.at = vb.make_positions(self.position, rows_per_seq=n_nodes, seq_rows=self.len)
        self.ws = torch.empty(vb.vg_tree_verify_workspace_size(self.dims, n_nodes), dtype=torch.uint8, device=dev)

    @staticmethod
    def _dense(name: str, t: torch.Tensor, dtype: torch.dtype, least: tuple, device) -> None:
        """Refuses a tensor that is not of that type and device, dense, and in each dimension at least as long."""
        if (t.dtype != dtype or t.device != device or not t.is_contiguous() or t.dim() != len(least)
                or any(n < m for n, m in zip(t.shape, least))):
            raise ValueError(f"{name}: dense {dtype} of at least {least} on {device}, not {t.dtype} {tuple(t.shape)} "
                             f"with strides {t.stride()} on {t.device}")

    def _rows(self, name: str, t: torch.Tensor, heads: int) -> None:
        """Refuses rows that the kernels cannot read: [B * n_nodes] of heads * d together, or [B][n_nodes] dense."""
        rows = self.B * self.n_nodes
        if t.dim() < 2 or t.numel() != rows * heads * self.d or t.shape[0] != rows or not t[0].is_contiguous():
            raise ValueError(f"{name}: {rows} rows of {heads} heads of {self.d} each together, not {tuple(t.shape)}")
        if t.dtype != torch.bfloat16 or t.device != self.visible.device:
            raise ValueError(f"{name}: bfloat16 on {self.visible.device}, not {t.dtype} on {t.device}")

    def build(self, stream=None) -> None:
        """Who attends whom, and the nodes' positions, from their parents."""
        vb.vg_tree_build(self.parent, self.n_nodes, self.len, self.B, self.n_nodes, self.prefix_len, self.visible,
                         self.position, dev_status=self.status, stream=stream)

    def rope_append(self, layer: int, rope: vb.vg_rope, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                    q_out: torch.Tensor | None = None, stream=None) -> None:
        """Rotate the nodes' q ([B * n_nodes][H_q][d], in place without q_out) and k at their positions; k and v
        enter the layer's cache behind the prefix."""
        q_out = q if q_out is None else q_out
        for name, t, heads in (("q", q, self.Hq), ("k", k, self.Hkv), ("v", v, self.Hkv), ("q_out", q_out, self.Hq)):
            self._rows(name, t, heads)
        vb.vg_rope_append_at(self.dims, self.cache[layer], rope, self.at, q, q.stride(0), k, k.stride(0), v, v.stride(0),
                             None, self.B * self.n_nodes, self.prefix_len, q_out, q_out.stride(0),
                             dev_status=self.status, stream=stream)

    def verify(self, layer: int, q: torch.Tensor, out: torch.Tensor, score_rows: torch.Tensor | None = None,
               scores: torch.Tensor | None = None, stream=None) -> None:
        """Attention of the nodes over prefix and ancestors (both in the cache).  With scores (float32 [B][max_len or more])
        the summed logits of the prefix, of the nodes that score_rows names (int64 [B][words], bits)."""
        for name, t in (("q", q), ("out", out)):
            self._rows(name, t, self.Hq)
            if not t.is_contiguous():
                raise ValueError(f"{name}: dense, not with strides {t.stride()}")
        if (score_rows is None) != (scores is None):
            raise ValueError("score_rows and scores: both or neither")
        if scores is not None:
            dev = self.visible.device
            self._dense("score_rows", score_rows.view(torch.int64) if score_rows.dtype == torch.uint64 else score_rows,
                        torch.int64, (self.B, self.words), dev)
            if score_rows.shape[1] != self.words:
                raise ValueError(f"score_rows: rows of {self.words} words, not {score_rows.shape[1]}")
            if (scores.dtype != torch.float32 or scores.device != dev or scores.dim() != 2 or scores.shape[0] < self.B
                    or scores.shape[1] < self.max_len or (scores.shape[1] > 1 and scores.stride(1) != 1)):
                raise ValueError(f"scores: {self.B} rows of float32, {self.max_len} or more together, on {dev}, not "
                                 f"{scores.dtype} {tuple(scores.shape)} with strides {scores.stride()} on {scores.device}")
        vb.vg_tree_verify_attn(self.dims, self.cache[layer], self.tree, q, None, None, self.prefix_len, score_rows, scores,
                               scores.stride(0) if scores is not None else 0, out, self.ws, dev_status=self.status,
                               stream=stream)

    def sample(self, logits: torch.Tensor, params: vb.vg_sampling, u: torch.Tensor, stream=None) -> None:
        """The target's token after every node, from its logits ([B * n_nodes][V] float32 or bfloat16).  params: a set
        for each sequence, rows_per_set = n_nodes and set_rows = len (or one for each node)."""
        rows = self.B * self.n_nodes
        dev = self.visible.device
        if (logits.dim() != 2 or logits.shape[0] != rows or logits.stride(1) != 1 or u.numel() != rows
                or not u.is_contiguous()):
            raise ValueError(f"logits of {rows} rows and as many dense u, not {tuple(logits.shape)} and {tuple(u.shape)} "
                             f"with strides {u.stride()}")
        for t in (logits, u, *(t for t in getattr(params, "tensors", ()) if t is not None)):
            if t.device != dev:
                raise ValueError(f"logits, u and params on {dev}, not {t.device}")
        if params.rows_per_set not in (self.n_nodes, 1):
            raise ValueError(f"params of {params.rows_per_set} rows a set: {self.n_nodes} (a sequence's nodes) or 1")
        kind = {torch.float32: vb.VG_LOGITS_FP32, torch.bfloat16: vb.VG_LOGITS_BF16}.get(logits.dtype)
        if kind is None or u.dtype != torch.float32:
            raise ValueError(f"logits in float32 or bfloat16 and u in float32, not {logits.dtype} and {u.dtype}")
        vb.vg_sample(logits, kind, logits.stride(0), rows, logits.shape[1], params, u, self.target, self.prob, None, 0,
                     self.ws, dev_status=self.status, stream=stream)

    def accept(self, stream=None) -> None:
        """The walk along ``target``: path, n_accept, next_token; the accepted rows move behind the prefix in every
        layer, and prefix_len advances."""
        vb.vg_tree_accept(self.dims, self.cache[0], self.caches, self.parent, self.n_nodes, self.len, self.n_nodes,
                          self.tokens, self.target, self.prefix_len, self.path, self.n_accept, self.next_token,
                          self.prefix_len, dev_status=self.status, stream=stream)

    def check_status(self) -> int:
        return int(self.status.item())


class IterationPlan:
    """An owned vg_iteration_plan.  It holds the tensors it was captured on, so they stay
    allocated at the same addresses for as long as the plan lives."""

    def __init__(self, handle: int, tensors: list):
        self.handle = handle
        self._tensors = tensors

    def launch(self, stream=None) -> None:
        if not self.handle:
            raise RuntimeError("the plan was closed")
        vb.vg_iteration_plan_launch(self.handle, stream)

    def close(self) -> None:
        if self.handle:
            vb.vg_iteration_plan_destroy(self.handle)
            self.handle = None
        self._tensors = []

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
