"""The operators around a paged batch, in their plain form and as the library's calls.

Four operators that a serving loop on this library's cache uses between its verification
steps, each as cases with inputs, one pass, its work and its definition in 64 bits:

* ``shared``  attention of the verify rows of a batch whose groups share a prefix, with the
              aggregated logits of every prefix entry;
* ``rope``    rotary positions of new q and k rows, and the append of k and v to the cache;
* ``pages``   the page pool: ``fork`` (children share a parent's pages, the last partial page
              copied), ``resize`` (rows freed and grown) and ``compact`` (live pages moved
              down to the front of the pool).

``own`` selects the side that ``run`` computes: elementary torch operations, or the
library's entry points.
"""
import math
import random

import torch

own = False

# ---------------------------------------------------------------- cases


def _shared(name, **kw):
    c = dict(op="shared", B=1, Hq=32, Hkv=8, d=128, gamma=0, groups=1, shared=1024, private_lo=1, private_hi=64,
             page=64, scores=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def _rope(name, **kw):
    c = dict(op="rope", B=1, Hq=32, Hkv=8, d=128, rows_lo=1, rows_hi=1, pos_lo=0, pos_hi=4096, page=64, rot=128,
             layout="half", scaling="plain", base=500000.0, factor=1.0, orig=8192)
    c.update(kw)
    return dict(c, name=name) if name else c


def _pages(name, op, **kw):
    c = dict(op=op, seqs=8, n=4, layers=1, page=16, tokens=2048, len_lo=1, len_hi=1024, room=8)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # two continuations of a short prompt on the small test heads: a step where only latency counts
        _shared("shared_tiny", B=2, Hq=8, Hkv=2, d=64, shared=512, private_lo=1, private_hi=40, page=16),
        # one token for each of 16 continuations of a long document: bound by reading the prefix once
        _shared("shared_decode_32k", B=16, shared=32768, private_lo=64, private_hi=512),
        # verification of 6 drafts in a ragged batch over three prompts of odd lengths, with the selection's logits
        _shared("shared_verify_groups", B=8, gamma=6, groups=3, shared=20011, private_lo=1, private_hi=2000, page=16,
                scores=True),
        # a large batch of samples from one prompt, 7 drafts verified: bound by the tensor cores
        _shared("shared_verify_b64", B=64, gamma=7, shared=16384, private_lo=100, private_hi=1000, scores=True),
        # the rows of one verification step, at far positions, frequencies scaled by parts
        _rope("rope_step", B=8, rows_lo=7, rows_hi=7, pos_lo=4096, pos_hi=65536, scaling="ramp", factor=8.0),
        # prompts of a ragged batch entering the cache, interleaved pairs in half of each head
        _rope("rope_prompts", B=8, rows_lo=600, rows_hi=4000, pos_lo=0, pos_hi=2000, rot=64, layout="interleaved",
              page=16),
        # four branches from one sequence, one layer's pages
        _pages("fork_4", "fork", seqs=8, n=4, len_lo=500, len_hi=1000),
        # 64 branches from 8 prompts over 16 layers
        _pages("fork_64_layers", "fork", seqs=128, n=64, layers=16, page=64, tokens=1024 * 64, len_lo=100, len_hi=2000),
        # a handful of sequences end and others begin
        _pages("resize_16", "resize", seqs=32, n=16, tokens=16384, len_lo=1, len_hi=900),
        # a pool of 131072 pages, 512 of 1024 sequences replaced
        _pages("resize_pool", "resize", seqs=1024, n=512, tokens=131072 * 16, len_lo=1, len_hi=3900),
        # a small pool's holes closed, one layer
        _pages("compact_small", "compact", seqs=16, n=8, tokens=4096, len_lo=1, len_hi=400),
        # holes closed over 8 layers of a pool of 1024 pages
        _pages("compact_layers", "compact", seqs=64, n=24, layers=8, page=64, tokens=1024 * 64, len_lo=64, len_hi=1900),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["shared", "shared", "rope", "fork", "resize", "compact"])
    if kind == "shared":
        Hq, Hkv, d = rng.choice([(32, 8, 128), (64, 8, 128), (8, 2, 64), (16, 1, 64), (40, 10, 128), (12, 3, 128)])
        B = _log(rng, 1, 64)
        gamma = rng.randint(0, min(7, 64 // (Hq // Hkv) - 1))
        cap = min(40000, 16384 * 64 * 8 * 32 // (B * (gamma + 1) * Hq))  # no more work than the largest listed case
        hi = _log(rng, 1, 1500)
        return _shared(None, B=B, Hq=Hq, Hkv=Hkv, d=d, gamma=gamma, groups=rng.randint(1, min(B, 5)),
                       shared=_log(rng, 40, max(64, cap)), private_lo=rng.randint(0, hi), private_hi=hi,
                       page=rng.choice([0, 8, 16, 32, 64, 128]) if B <= 16 else rng.choice([8, 16, 32, 64, 128]),
                       scores=rng.random() < 0.6)
    if kind == "rope":
        Hq, Hkv, d = rng.choice([(32, 8, 128), (64, 8, 128), (8, 2, 64), (16, 1, 64), (40, 10, 128)])
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, max(2, 24000 // B))
        return _rope(None, B=B, Hq=Hq, Hkv=Hkv, d=d, rows_lo=rng.randint(0, hi), rows_hi=hi, pos_lo=0,
                     pos_hi=_log(rng, 1, max(2, 500000 // B)), page=rng.choice([0, 1, 5, 16, 64]),
                     rot=rng.choice([d, d // 2, d // 4, 2 * rng.randint(1, d // 2)]),
                     layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["plain", "linear", "base", "ramp"]),
                     base=rng.choice([10000.0, 500000.0, 1000000.0]), factor=rng.choice([2.0, 8.0, 32.0]), orig=8192)
    layers = _log(rng, 1, 8)
    page = rng.choice([1, 5, 16, 64, 128])
    hi = _log(rng, 2, 1000)
    seqs = _log(rng, 4, 64)
    tokens = seqs * (-(-(hi + 16) // page) + 1) * page * 2
    return _pages(None, kind, seqs=seqs, n=rng.randint(1, max(1, seqs // 2)), layers=layers if kind != "resize" else 1,
                  page=page, tokens=tokens, len_lo=rng.randint(1, hi), len_hi=hi, room=rng.randint(0, 16))


# ---------------------------------------------------------------- lengths (of a case, not of a seed: work() counts them)


def _lengths(case):
    r = random.Random(20)
    if case["op"] == "shared":
        B, ng = case["B"], case["groups"]
        cuts = sorted(r.sample(range(1, B), ng - 1)) if ng > 1 else []
        start = [0] + cuts + [B]
        shared = [case["shared"]] + [max(1, int(case["shared"] * r.uniform(0.3, 1.0))) for _ in range(ng - 1)]
        n = [shared[j] + r.randint(case["private_lo"], case["private_hi"]) for j in range(ng) for _ in range(start[j + 1] - start[j])]
        return start, shared, n
    if case["op"] == "rope":
        rows = [r.randint(case["rows_lo"], case["rows_hi"]) for _ in range(case["B"])]
        rows[0] = max(1, rows[0])
        return rows, [r.randint(case["pos_lo"], case["pos_hi"]) for _ in range(case["B"])]
    return [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]


def _pages_of(tokens, page):
    return -(-tokens // page)


def work(case):
    op = case["op"]
    if op == "shared":
        start, shared, n = _lengths(case)
        R, Hq, Hkv, d = case["gamma"] + 1, case["Hq"], case["Hkv"], case["d"]
        rows = case["B"] * R * Hq
        own_tokens = [n[b] - shared[j] for j in range(len(shared)) for b in range(start[j], start[j + 1])]
        tokens = sum(shared) + sum(own_tokens) + case["B"] * R
        keys = sum(n)
        return {"bytes": tokens * Hkv * d * 2 * 2 + 2 * rows * d * 2 + (4 * keys if case["scores"] else 0),
                "flops": 4 * R * Hq * d * (keys + case["B"] * (R + 1) / 2) + (2 * Hkv * d * keys if case["scores"] else 0)}
    if op == "rope":
        rows, _ = _lengths(case)
        heads = case["Hq"] + 2 * case["Hkv"]
        return {"bytes": 2 * sum(rows) * heads * case["d"] * 2, "flops": sum(rows) * (case["Hq"] + case["Hkv"]) * case["rot"] * 3}
    st = _plan(case)
    token = _ROW * 2
    table = 4 * len(st["refs"])
    if op == "fork":
        moved = sum(st["length"][j] % case["page"] for j in range(case["n"]))
        return {"bytes": 2 * moved * 2 * case["layers"] * token + table, "flops": 0}
    if op == "resize":
        touched = sum(_pages_of(x, case["page"]) for x in st["target"])
        return {"bytes": table + 8 * touched, "flops": 0}
    live = sum(1 for x in st["refs"] if x > 0)
    moves = sum(1 for x in st["refs"][live:] if x > 0)
    held = sum(st["held"])
    return {"bytes": 2 * moves * case["page"] * 2 * case["layers"] * token + 2 * table + 8 * held, "flops": 0}


# ---------------------------------------------------------------- the page pool's plan (host integers)

_ROW = 8 * 128  # elements of a token's keys of all heads, as in the 8-head layers


def _plan(case):
    """Sequences holding scattered pages of a pool, and the request: what a running server has."""
    r = random.Random(31)
    lens, page, n = _lengths(case), case["page"], case["n"]
    room = case["room"]
    most = max(_pages_of(max(lens) + room, page), 1)
    n_pages = max(case["tokens"] // page, 1)
    order = list(range(n_pages))
    r.shuffle(order)
    # the last n sequences are the ones that a request replaces; the others stay
    held = [_pages_of(lens[s], page) for s in range(case["seqs"])]
    table, at = [], 0
    for s in range(case["seqs"]):
        if at + held[s] > n_pages * 3 // 4:
            held[s] = 0
        table.append(order[at:at + held[s]] + [-1] * (most - held[s]))
        at += held[s]
    refs = [0] * n_pages
    for s in range(case["seqs"]):
        for p in table[s][:held[s]]:
            refs[p] += 1
    out = dict(table=table, held=held, refs=refs, lens=lens, most=most, n_pages=n_pages)
    if case["op"] == "fork":
        parents = [s for s in range(case["seqs"] - n) if held[s] > 0][:8]
        out["child"] = list(range(case["seqs"] - n, case["seqs"]))
        out["parent"] = [parents[j % len(parents)] for j in range(n)]
        out["length"] = [min(lens[out["parent"][j]], r.randint(max(1, lens[out["parent"][j]] - 40), lens[out["parent"][j]])) for j in range(n)]
    if case["op"] == "resize":
        seq = list(range(case["seqs"]))
        r.shuffle(seq)
        out["seq"] = seq[:n]
        out["target"] = [r.randint(1, max(lens)) for _ in range(n)]
        free = n_pages - sum(held[s] for s in seq[n:])
        while sum(_pages_of(x, page) for x in out["target"]) > free:
            out["target"] = [max(1, x // 2) for x in out["target"]]
    if case["op"] == "compact":  # n sequences ended since: their pages are the holes
        for s in r.sample(range(case["seqs"]), n):
            for p in table[s][:held[s]]:
                refs[p] -= 1
            table[s] = [-1] * most
            held[s] = 0
    return out


# ---------------------------------------------------------------- inputs


def _normal(gen, shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op == "shared":
        start, shared, n = _lengths(case)
        B, R, Hq, Hkv, d, page = case["B"], case["gamma"] + 1, case["Hq"], case["Hkv"], case["d"], case["page"]
        u = torch.randn(d, generator=gen, device="cuda")
        u /= u.norm()
        if page:
            W = max(_pages_of(x + R, page) for x in n)
            total = sum(s // page for s in shared)
            rows, at = [], 0
            for j in range(len(shared)):
                common = list(range(at, at + shared[j] // page))
                at += len(common)
                for b in range(start[j], start[j + 1]):
                    mine = _pages_of(n[b] + R, page) - len(common)
                    rows.append(common + list(range(at, at + mine)) + [0] * (W - len(common) - mine))
                    at += mine
            total = at
            perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
            st["page_table"] = perm[_ints(rows, torch.int64)].contiguous()
            slots = total * page
            st["seq_offset"] = None
        else:
            off = [0]
            for b in range(B):
                off.append(off[-1] + _pages_of(n[b] + R, 16) * 16)
            slots = off[-1]
            st["page_table"] = None
            st["seq_offset"] = _ints(off[:-1], torch.int64)
        K, V = _normal(gen, (slots, Hkv, d)), _normal(gen, (slots, Hkv, d))
        heavy = torch.rand(slots, generator=gen, device="cuda") < 0.02  # 2 % of the keys lie along one direction
        K = torch.where(heavy[:, None, None], (3 * u + 0.5 * K.float()).to(torch.bfloat16), K)
        if page:  # the tokens of a shared prefix past its last full page are each sequence's own copy
            table = st["page_table"].long()
            for j in range(len(shared)):
                rem, pi = shared[j] % page, shared[j] // page
                for b in range(start[j] + 1, start[j + 1]):
                    if rem:
                        x, y = int(table[b, pi]) * page, int(table[start[j], pi]) * page
                        K[x:x + rem], V[x:x + rem] = K[y:y + rem], V[y:y + rem]
        else:
            for j in range(len(shared)):
                for b in range(start[j] + 1, start[j + 1]):
                    K[off[b]:off[b] + shared[j]] = K[off[start[j]]:off[start[j]] + shared[j]]
                    V[off[b]:off[b] + shared[j]] = V[off[start[j]]:off[start[j]] + shared[j]]
        q = (torch.randn((B, R, Hq, d), generator=gen, device="cuda") + 6 * u).to(torch.bfloat16)
        st.update(K=K, V=V, q=q, prefix_len=_ints(n), group_start=_ints(start), shared_len=_ints(shared), max_len=max(n))
        stride = _pages_of(max(n), 4) * 4
        st.update(stride=stride, out=torch.empty_like(q), mask=(1 | 1 << (R - 1)),
                  scores=torch.zeros((B, stride), device="cuda") if case["scores"] else None)
    elif op == "rope":
        rows, pos = _lengths(case)
        B, Hq, Hkv, d, page = case["B"], case["Hq"], case["Hkv"], case["d"], case["page"]
        row_start = [0]
        for x in rows:
            row_start.append(row_start[-1] + x)
        N = row_start[-1]
        st["qkv"] = _normal(gen, (N, (Hq + 2 * Hkv) * d))  # one projection's output: q, k, v side by side
        need = [_pages_of(p + x, page or 1) for p, x in zip(pos, rows)]
        if page:
            # only the pages of the new rows exist here: the rest of each row is another layer's concern
            W = max(max(need), 1)
            first = [p // page for p in pos]
            table, at = [], 0
            for b in range(B):
                table.append([0] * first[b] + list(range(at, at + need[b] - first[b])) + [0] * (W - need[b]))
                at += need[b] - first[b]
            perm = torch.randperm(max(at, 1), generator=gen, device="cuda").to(torch.int32)
            st["page_table"] = perm[_ints(table, torch.int64)].contiguous()
            st["seq_offset"] = None
            slots = max(at, 1) * page
        else:
            off = [0]
            for b in range(B):
                off.append(off[-1] + need[b] + 3)
            slots = off[-1]
            st["page_table"] = None
            st["seq_offset"] = _ints(off[:-1], torch.int64)
        st.update(K=torch.zeros((slots, Hkv, d), device="cuda", dtype=torch.bfloat16),
                  V=torch.zeros((slots, Hkv, d), device="cuda", dtype=torch.bfloat16),
                  row_start=_ints(row_start), prefix_len=_ints(pos), rows=N, max_len=max(pos),
                  q_out=torch.empty((N, Hq, d), device="cuda", dtype=torch.bfloat16),
                  inv=torch.tensor(_inverse(case), dtype=torch.float64, device="cuda"), mscale=_mscale(case))
    else:
        p = _plan(case)
        slots = p["n_pages"] * case["page"]
        st.update(table=_ints(p["table"]), held=_ints(p["held"]), refs=_ints(p["refs"]), n_pages=p["n_pages"])
        if op == "resize":
            salt = torch.randperm(case["n"], generator=gen, device="cuda")  # which request grows to which length
            st.update(seq=_ints(p["seq"]), target=_ints(p["target"])[salt].contiguous(), none=_ints([0] * case["n"]))
        else:
            st["KV"] = _normal(gen, (case["layers"], 2, slots, _ROW))
        if op == "fork":
            st.update(parent=_ints(p["parent"]), child=_ints(p["child"]), length=_ints(p["length"]))
        if op == "compact":
            st.update(table_out=torch.empty_like(st["table"]), refs_out=torch.empty_like(st["refs"]),
                      n_live=torch.zeros(1, dtype=torch.int32, device="cuda"))
    return st


def _inverse(case):
    """Radians per position of each rotated pair."""
    rot, base, factor = case["rot"], case["base"], case["factor"]
    if case["scaling"] == "base" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    inv = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        inv = [f / factor for f in inv]
    if case["scaling"] == "ramp":
        keep = [min(1.0, max(0.0, (case["orig"] * f / (2 * math.pi) - 1.0) / 31.0)) for f in inv]
        inv = [f * (w + (1 - w) / factor) for f, w in zip(inv, keep)]
    return inv


def _mscale(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "ramp" else 1.0


# ---------------------------------------------------------------- plain forms


def _slots(st, tokens):
    """Cache slot of each sequence's token positions ([B, n])."""
    page = st["case"]["page"]
    if not page:
        return st["seq_offset"][:, None] + tokens
    at = (tokens // page).clamp(max=st["page_table"].shape[1] - 1)
    return torch.gather(st["page_table"].long(), 1, at) * page + tokens % page


def _plain_shared(st):
    c = st["case"]
    B, R, Hq, Hkv, d = c["B"], c["gamma"] + 1, c["Hq"], c["Hkv"], c["d"]
    G = Hq // Hkv
    n = st["prefix_len"].long()
    L = st["max_len"] + R
    j = torch.arange(L, device="cuda")
    slots = _slots(st, j.expand(B, L).minimum(n[:, None] + R - 1))
    K, V = st["K"][slots].float(), st["V"][slots].float()  # [B, L, Hkv, d]
    q = st["q"].float().view(B, R, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * G, d)
    s = (q @ K.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(d))
    last = (n[:, None] + torch.arange(R, device="cuda")).repeat_interleave(G, 1)  # a row's own position
    s = torch.where(j <= last[:, None, :, None], s, float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = (p @ V.permute(0, 2, 1, 3)) / p.sum(-1, keepdim=True)
    out = o.view(B, Hkv, R, G, d).permute(0, 2, 1, 3, 4).reshape(B, R, Hq, d).to(torch.bfloat16)
    if not c["scores"]:
        return {"out": out}
    rows = st["q"].float()[:, sorted({0, R - 1})].sum(1).view(B, Hkv, G, d).sum(2).reshape(B, Hkv * d, 1)
    sc = (K.reshape(B, L, Hkv * d) @ rows).squeeze(-1)[:, :st["max_len"]] * (1.0 / math.sqrt(d))
    sc = torch.where(j[:st["max_len"]] < n[:, None], sc, 0.0)
    return {"out": out, "scores": torch.nn.functional.pad(sc, (0, st["stride"] - st["max_len"]))}


def _plain_rope(st):
    c = st["case"]
    Hq, Hkv, d, rot, N = c["Hq"], c["Hkv"], c["d"], c["rot"], st["rows"]
    r = torch.arange(N, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(st["row_start"], r, right=True) - 1
    pos = (st["prefix_len"] - st["row_start"][:-1])[b].long() + r
    angle = pos[:, None].double() * st["inv"]
    cos = (torch.cos(angle) * st["mscale"]).float()[:, None]
    sin = (torch.sin(angle) * st["mscale"]).float()[:, None]

    def turn(x):  # [N, H, d]
        x, rest = x[..., :rot].float(), x[..., rot:]
        if c["layout"] == "half":
            a, e = x[..., :rot // 2], x[..., rot // 2:]
            y = torch.cat((a * cos - e * sin, a * sin + e * cos), -1)
        else:
            a, e = x[..., 0::2], x[..., 1::2]
            y = torch.stack((a * cos - e * sin, a * sin + e * cos), -1).flatten(-2)
        return torch.cat((y.to(torch.bfloat16), rest), -1)

    q, k, v = st["qkv"].split((Hq * d, Hkv * d, Hkv * d), 1)
    if c["page"]:
        slot = st["page_table"][b, pos // c["page"]].long() * c["page"] + pos % c["page"]
    else:
        slot = st["seq_offset"][b] + pos
    st["K"][slot] = turn(k.reshape(N, Hkv, d))
    st["V"][slot] = v.reshape(N, Hkv, d)
    return {"q": turn(q.reshape(N, Hq, d)), "K": st["K"], "V": st["V"]}


def _release(table, held, refs, seq, keep):
    """References of `seq`'s pages past `keep` given back; the touched rows of the table."""
    i = torch.arange(table.shape[1], device="cuda")
    rows = table[seq.long()]
    drop = (i < held[seq.long()][:, None]) & (i >= keep[:, None])
    more = torch.cat((refs, refs.new_zeros(1)))  # the last entry takes what drops nothing
    more.index_add_(0, torch.where(drop, rows, refs.shape[0]).reshape(-1).long(), torch.full((rows.numel(),), -1, dtype=refs.dtype, device="cuda"))
    refs.copy_(more[:-1])
    return torch.where(drop, -1, rows), i


def _take(refs, have, total, rows, i):
    """Pages [have, total) of each row from the lowest free pages, in order."""
    need = total - have
    first = torch.cumsum(need, 0) - need
    free = torch.argsort((refs > 0).to(torch.int8), stable=True).to(torch.int32)
    new = (i >= have[:, None]) & (i < total[:, None])
    rank = (first[:, None] + i - have[:, None]).clamp(0, refs.shape[0] - 1)
    rows = torch.where(new, free[rank], rows)
    more = torch.cat((refs, refs.new_zeros(1)))
    more.index_add_(0, torch.where(new, rows, refs.shape[0]).reshape(-1).long(), torch.ones(rows.numel(), dtype=refs.dtype, device="cuda"))
    refs.copy_(more[:-1])
    return rows, free, first


def _plain_resize(st):
    page = st["case"]["page"]
    for length in (st["none"], st["target"]):
        seq = st["seq"].long()
        total = (length + page - 1) // page
        rows, i = _release(st["table"], st["held"], st["refs"], seq, total)
        rows, _, _ = _take(st["refs"], torch.minimum(st["held"][seq], total), total, rows, i)
        st["table"][seq] = rows
        st["held"][seq] = total
    return {"table": st["table"], "held": st["held"], "refs": st["refs"]}


def _plain_fork(st):
    c = st["case"]
    page, room = c["page"], c["room"]
    parent, child, length = st["parent"].long(), st["child"].long(), st["length"]
    full, total = length // page, (length + room + page - 1) // page
    rows, i = _release(st["table"], st["held"], st["refs"], child, torch.zeros_like(length))
    theirs = st["table"][parent]
    share = i < full[:, None]
    rows = torch.where(share, theirs, rows)
    rows, free, first = _take(st["refs"], full, total, rows, i)
    more = torch.cat((st["refs"], st["refs"].new_zeros(1)))
    more.index_add_(0, torch.where(share, theirs, st["n_pages"]).reshape(-1).long(), torch.ones(theirs.numel(), dtype=torch.int32, device="cuda"))
    st["refs"].copy_(more[:-1])
    st["table"][child] = rows
    st["held"][child] = total
    # the tokens of the last page that the child has in part; the others copy a parent's slot onto itself
    t = torch.arange(page, device="cuda")
    part = t < (length % page)[:, None]
    at = full.clamp(max=rows.shape[1] - 1).long()[:, None]
    here = theirs[:, :1].long() * page + t
    src = torch.where(part, theirs.gather(1, at).long() * page + t, here).reshape(-1)
    dst = torch.where(part, rows.gather(1, at).long() * page + t, here).reshape(-1)
    st["KV"].index_copy_(2, dst, st["KV"].index_select(2, src))
    return {"table": st["table"], "held": st["held"], "refs": st["refs"], "KV": st["KV"]}


def _plain_compact(st):
    c = st["case"]
    live = st["refs"] > 0
    n_live = live.sum().to(torch.int32)
    i = torch.arange(st["n_pages"], device="cuda", dtype=torch.int32)
    holes = (~live & (i < n_live)).nonzero().squeeze(1)
    movers = (live & (i >= n_live)).nonzero().squeeze(1)
    to = i.clone()
    to[movers] = holes.to(torch.int32)
    held = torch.arange(st["table"].shape[1], device="cuda") < st["held"][:, None]
    table = torch.where(held, to[st["table"].clamp(min=0).long()], st["table"])
    refs = st["refs"].clone()
    refs[holes] = st["refs"][movers]
    refs[movers] = 0
    kv = st["KV"].view(c["layers"], 2, st["n_pages"], c["page"] * _ROW)
    kv.index_copy_(2, holes, kv.index_select(2, movers))
    return {"table": table, "refs": refs, "n_live": n_live.view(1), "KV": st["KV"]}


# ---------------------------------------------------------------- the library's calls


def _own(st):
    from self_speculative_sparse_gb300 import binding as vb

    c = st["case"]
    op = c["op"]
    if op in ("shared", "rope") and "dims" not in st:
        st["dims"] = vb.make_dims(c["B"], c["Hq"], c["Hkv"], c["d"], c.get("gamma", 0), st["max_len"])
        st["cache"] = vb.make_cache(st["K"], st["V"], st["seq_offset"], page_table=st["page_table"], page_size=c["page"])
    if op == "shared":
        if "ws" not in st:
            st["groups"] = vb.make_groups(st["group_start"], st["shared_len"])
            st["ws"] = torch.empty(vb.vg_shared_verify_workspace_size(st["dims"], st["groups"]), dtype=torch.uint8, device="cuda")
        vb.vg_shared_verify_attn(st["dims"], st["cache"], st["groups"], st["q"], None, None, st["prefix_len"],
                                 st["mask"] if c["scores"] else 0, st["scores"], st["stride"], st["out"], st["ws"])
        return {"out": st["out"], "scores": st["scores"]} if c["scores"] else {"out": st["out"]}
    if op == "rope":
        if "rope" not in st:
            kind = {"plain": vb.VG_ROPE_PLAIN, "linear": vb.VG_ROPE_LINEAR, "base": vb.VG_ROPE_BASE, "ramp": vb.VG_ROPE_RAMP}[c["scaling"]]
            st["freq"] = torch.from_numpy(vb.vg_rope_freqs(c["rot"], c["base"], kind, c["factor"], c["orig"], 1.0, 32.0).view("int64")).cuda()
            st["rope"] = vb.make_rope(st["freq"], c["rot"], vb.VG_ROPE_HALF if c["layout"] == "half" else vb.VG_ROPE_INTERLEAVED, st["mscale"])
        qd, kd = c["Hq"] * c["d"], c["Hkv"] * c["d"]
        at, w = st["qkv"].data_ptr(), qd + 2 * kd
        vb.vg_rope_append(st["dims"], st["cache"], st["rope"], at, w, at + 2 * qd, w, at + 2 * (qd + kd), w,
                          st["row_start"], st["rows"], st["prefix_len"], st["q_out"], qd)
        return {"q": st["q_out"], "K": st["K"], "V": st["V"]}
    if "pool" not in st:
        st["pool"] = vb.make_pages(st["table"], st["held"], st["refs"], c["page"])
        st["ws"] = torch.empty(vb.vg_pages_workspace_size(st["pool"]), dtype=torch.uint8, device="cuda")
        if op != "resize":
            st["caches"] = vb.make_caches([(st["KV"][x, 0], st["KV"][x, 1]) for x in range(c["layers"])])
    if op == "resize":
        vb.vg_pages_resize(st["pool"], st["seq"], st["none"], c["n"], st["ws"])
        vb.vg_pages_resize(st["pool"], st["seq"], st["target"], c["n"], st["ws"])
        return {"table": st["table"], "held": st["held"], "refs": st["refs"]}
    if op == "fork":
        vb.vg_pages_fork(st["pool"], st["caches"], _ROW * 2, st["parent"], st["child"], st["length"], c["n"], c["room"], st["ws"])
        return {"table": st["table"], "held": st["held"], "refs": st["refs"], "KV": st["KV"]}
    vb.vg_pages_compact(st["pool"], st["caches"], _ROW * 2, st["table_out"], st["refs_out"], st["n_live"], st["ws"])
    return {"table": st["table_out"], "refs": st["refs_out"], "n_live": st["n_live"], "KV": st["KV"]}


def run(state):
    if own:
        return _own(state)
    return {"shared": _plain_shared, "rope": _plain_rope, "fork": _plain_fork, "resize": _plain_resize,
            "compact": _plain_compact}[state["case"]["op"]](state)


# ---------------------------------------------------------------- definitions in 64 bits


def _exact_shared(st):
    c = st["case"]
    B, R, Hq, Hkv, d = c["B"], c["gamma"] + 1, c["Hq"], c["Hkv"], c["d"]
    G = Hq // Hkv
    out = torch.zeros((B, R, Hq, d), dtype=torch.float64, device="cuda")
    scores = torch.zeros((B, st["stride"]), dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["prefix_len"].tolist()):
        i = torch.arange(n + R, device="cuda")
        if c["page"]:
            slot = st["page_table"][b].long()[i // c["page"]] * c["page"] + i % c["page"]
        else:
            slot = i + st["seq_offset"][b]
        K, V = st["K"][slot].double(), st["V"][slot].double()
        for g in range(Hkv):
            q = st["q"][b, :, g * G:(g + 1) * G].double().reshape(R * G, d)
            s = torch.mm(q, K[:, g].t()) / math.sqrt(d)
            scores[b, :n] += s.view(R, G, -1)[sorted({0, R - 1})].sum((0, 1))[:n]
            for t in range(R):
                s[t * G:(t + 1) * G, n + t + 1:] = float("-inf")
            out[b, :, g * G:(g + 1) * G] = torch.mm(torch.softmax(s, 1), V[:, g]).view(R, G, d)
    return {"out": out, "scores": scores} if c["scores"] else {"out": out}


def _exact_rope(st):
    c = st["case"]
    Hq, Hkv, d, rot = c["Hq"], c["Hkv"], c["d"], c["rot"]
    inv = torch.tensor(_inverse(c), dtype=torch.float64, device="cuda")
    x = st["qkv"].double().view(st["rows"], Hq + 2 * Hkv, d)
    K, V = st["K"].double(), st["V"].double()
    y = x.clone()
    starts, before = st["row_start"].tolist(), st["prefix_len"].tolist()
    half = c["layout"] == "half"
    first = torch.arange(rot // 2, device="cuda") * (1 if half else 2)
    second = first + (rot // 2 if half else 1)
    for b in range(c["B"]):
        lo, hi = starts[b], starts[b + 1]
        if lo == hi:
            continue
        pos = torch.arange(before[b], before[b] + hi - lo, device="cuda")
        z = torch.polar(torch.full((hi - lo, rot // 2), st["mscale"], dtype=torch.float64, device="cuda"), pos.double()[:, None] * inv)
        w = torch.complex(x[lo:hi, :Hq + Hkv, first], x[lo:hi, :Hq + Hkv, second]) * z[:, None]
        y[lo:hi, :Hq + Hkv, first], y[lo:hi, :Hq + Hkv, second] = w.real, w.imag
        if c["page"]:
            slot = st["page_table"][b].long()[pos // c["page"]] * c["page"] + pos % c["page"]
        else:
            slot = pos + st["seq_offset"][b]
        K[slot], V[slot] = y[lo:hi, Hq:Hq + Hkv], y[lo:hi, Hq + Hkv:]
    return {"q": y[:, :Hq].contiguous(), "K": K, "V": V}


def _exact_pages(st):
    c = st["case"]
    page = c["page"]
    table, held, refs = st["table"].tolist(), st["held"].tolist(), st["refs"].tolist()

    def drop(s, keep):
        for i in range(keep, held[s]):
            refs[table[s][i]] -= 1
            table[s][i] = -1
        held[s] = min(held[s], keep)

    def grow(s, total):
        for i in range(held[s], total):
            while refs[lowest[0]] > 0:
                lowest[0] += 1
            table[s][i] = lowest[0]
            refs[lowest[0]] = 1
        held[s] = total

    KV = st.get("KV")
    if c["op"] == "resize":
        seq = st["seq"].tolist()
        for s in seq:
            drop(s, 0)
        lowest = [0]
        for s, x in zip(seq, st["target"].tolist()):
            grow(s, -(-x // page))
        return {"table": torch.tensor(table), "held": torch.tensor(held), "refs": torch.tensor(refs)}
    if c["op"] == "fork":
        child = st["child"].tolist()
        for s in child:
            drop(s, 0)
        lowest, src, dst = [0], [], []
        for s, f, x in zip(child, st["parent"].tolist(), st["length"].tolist()):
            for i in range(x // page):
                table[s][i] = table[f][i]
                refs[table[f][i]] += 1
            held[s] = x // page
            grow(s, -(-(x + c["room"]) // page))
            for t in range(x % page):
                src.append(table[f][x // page] * page + t)
                dst.append(table[s][x // page] * page + t)
        if src:
            KV[:, :, torch.tensor(dst, device="cuda")] = KV[:, :, torch.tensor(src, device="cuda")]
        return {"table": torch.tensor(table), "held": torch.tensor(held), "refs": torch.tensor(refs), "KV": KV}
    live = sum(x > 0 for x in refs)
    to, hole = {}, 0
    for p in range(live, len(refs)):
        if refs[p] > 0:
            while refs[hole] > 0:
                hole += 1
            to[p], refs[hole], refs[p] = hole, refs[p], 0
    for s in range(len(table)):
        table[s] = [to.get(x, x) if i < held[s] else x for i, x in enumerate(table[s])]
    pages = KV.view(c["layers"], 2, st["n_pages"], -1)
    for p, h in to.items():
        pages[:, :, h] = pages[:, :, p]
    return {"table": torch.tensor(table), "refs": torch.tensor(refs), "n_live": torch.tensor([live]), "KV": KV}


def exact(case, seed):
    st = prepare(case, seed)
    return {"shared": _exact_shared, "rope": _exact_rope}.get(case["op"], _exact_pages)(st)
