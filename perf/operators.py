"""The paged-cache operators: what is measured, in plain form and as a user calls them.

A serving program packs the prompts of a step behind one another, keeps keys
and values in a pool of fixed-size pages that a table maps to sequences, and
shares pages between sequences that begin alike.  Five operators:

  prefill_packed  prompts of different lengths in one call, no cache
  prefill_paged   chunks of prompts on top of what their pages hold already
  decode_paged    one new token per sequence over its pages
  fork            sequences forked, then grown by a token (copy on write)
  compact         ended sequences freed, the pool compacted, new ones admitted

Attention is softmax(q k^T / 16) v times sigmoid(gate) per query head, causal
or within a sliding window, head size 256, rotary positions on the first
rot_dim dims.  Keys live rotated and in bf16 (that is what a page holds), and
the attention of a prompt reads them as its later decode steps will.

`own` false: elementary torch operations in 32 bits.  `own` true: the calls of
full_gqa_attention_gb300.
"""
from __future__ import annotations

import math
import random

import torch

own = False

D = 256
KINDS = {"full": (5e6, 64), "sliding": (1e4, 256)}   # RoPE base, rotated dims
DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a few short questions answered at once by the small model: latency
        dict(name="packed_short_sliding", op="prefill_packed", H=8, Hkv=2, kind="sliding",
             window=512, seqs=7, idle=1, longest=96, pad=5, mix=11),
        # a step's worth of chat prompts of every length
        dict(name="packed_mixed_full", op="prefill_packed", H=16, Hkv=4, kind="full", window=0,
             seqs=24, idle=2, longest=4096, pad=37, mix=12),
        # a document and its companions
        dict(name="packed_long_full", op="prefill_packed", H=16, Hkv=4, kind="full", window=0,
             seqs=4, idle=0, longest=20011, pad=0, mix=13),
        # prompts cut in chunks, on top of long cached prefixes
        dict(name="paged_chunks_full", op="prefill_paged", H=16, Hkv=4, kind="full", window=0,
             seqs=8, idle=2, longest=2048, prefix=24576, page=64, pad=0, mix=34),
        # follow-up turns through a sliding layer with small pages
        dict(name="paged_turns_sliding", op="prefill_paged", H=8, Hkv=2, kind="sliding",
             window=512, seqs=16, idle=3, longest=700, prefix=4096, page=16, pad=9, mix=15),
        # one user, a short chat: latency
        dict(name="decode_one_short", op="decode_paged", H=8, Hkv=2, kind="full", window=0,
             seqs=1, idle=0, longest=701, page=16, mix=16),
        # a serving batch with sequences of every length and idle slots
        dict(name="decode_ragged", op="decode_paged", H=16, Hkv=4, kind="full", window=0,
             seqs=48, idle=5, longest=16384, page=64, mix=17),
        # one very long context, larger than the L2 cache by far
        dict(name="decode_long", op="decode_paged", H=16, Hkv=4, kind="full", window=0, seqs=1,
             idle=0, longest=262139, page=128, mix=18),
        # two branches of a short chat: latency
        dict(name="fork_pair", op="fork", Hkv=2, layers=7, parents=1, copies=1, longest=300,
             page=16, mix=19),
        # sampling several answers to every prompt of a batch, the 4B model's nine full layers
        dict(name="fork_answers", op="fork", Hkv=4, layers=9, parents=32, copies=3, longest=1024,
             page=64, mix=20),
        # a handful of sequences end in a small pool: latency
        dict(name="compact_small", op="compact", Hkv=2, layers=7, rows=6, longest=200, page=16,
             mix=21),
        # half of a busy pool ends and the other half closes the gaps
        dict(name="compact_busy", op="compact", Hkv=4, layers=9, rows=24, longest=4096, page=64,
             mix=22),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill_packed", "prefill_paged", "decode_paged", "fork", "compact"])
    H, Hkv = rng.choice([(16, 4), (8, 2), (4, 4), (8, 4), (8, 1)])
    kind = rng.choice(["full", "sliding"])
    window = _log(rng, 32, 1024) if kind == "sliding" else 0
    page = rng.choice([16, 32, 64, 128, 256])
    c = dict(op=op, mix=rng.randrange(1 << 30))
    if op == "prefill_packed":
        longest = _log(rng, 16, 12000)
        seqs = _log(rng, 1, max(1, min(48, 60000 // longest)))
        c.update(H=H, Hkv=Hkv, kind=kind, window=window, seqs=seqs, idle=rng.randrange(3),
                 longest=longest, pad=rng.randrange(70))
    elif op == "prefill_paged":
        longest = _log(rng, 1, 3000)
        prefix = _log(rng, 1, 24000)
        seqs = _log(rng, 1, max(1, min(32, 60000 // (longest + prefix))))
        c.update(H=H, Hkv=Hkv, kind=kind, window=window, seqs=seqs, idle=rng.randrange(3),
                 longest=longest, prefix=prefix, page=page, pad=rng.randrange(70))
    elif op == "decode_paged":
        longest = _log(rng, 1, 131072)
        seqs = _log(rng, 1, max(1, min(192, 262144 // longest)))
        c.update(H=H, Hkv=Hkv, kind=kind, window=window, seqs=seqs, idle=rng.randrange(4),
                 longest=longest, page=page)
    elif op == "fork":
        c.update(Hkv=Hkv, layers=rng.randrange(1, 10), parents=_log(rng, 1, 24),
                 copies=rng.randrange(1, 4), longest=_log(rng, 1, 1024), page=page)
    else:
        c.update(Hkv=Hkv, layers=rng.randrange(1, 10), rows=2 * _log(rng, 1, 12),
                 longest=_log(rng, 1, 3500), page=page)
    return c


def _spread(mix, n, hi):
    """n lengths: one of them the longest, the others spread over [1, hi] by their logarithm."""
    rng = random.Random(mix)
    v = [hi] + [_log(rng, 1, hi) for _ in range(n - 1)]
    rng.shuffle(v)
    return v


def _plan(case):
    """Per sequence: new tokens and tokens cached before them; None in idle slots."""
    rng = random.Random(case["mix"] + 1)
    new = _spread(case["mix"], case["seqs"], case["longest"])
    if case["op"] == "prefill_paged":
        old = _spread(case["mix"] + 2, case["seqs"], case["prefix"])
        old = [0 if rng.random() < 0.2 and case["seqs"] > 1 else x for x in old]
    else:
        old = [0] * len(new)
    if case["op"] == "decode_paged":
        new, old = [1] * len(new), new
    rows = list(zip(new, old))
    for _ in range(case["idle"]):
        rows.insert(rng.randrange(len(rows) + 1), None)
    return rows


def _pairs(case, new, old):
    """Visible (query, key) pairs of `new` queries after `old` cached tokens."""
    w = case["window"] if case["kind"] == "sliding" else 1 << 40
    full = max(0, old + new - max(old, w))               # queries with a full window
    part = new - full                                    # queries that see old+1, old+2, ... keys
    return full * w + part * (2 * old + part + 1) // 2


def _first_key(case, old):
    return max(0, old - case["window"] + 1) if case["kind"] == "sliding" else 0


def work(case):
    op = case["op"]
    if op in ("fork", "compact"):
        moved, small = _page_work(case)
        page_bytes = case["layers"] * case["Hkv"] * case["page"] * D * 2 * 2
        return {"bytes": 2 * moved * page_bytes + small, "flops": 0}
    H, Hkv = case["H"], case["Hkv"]
    rows = [r for r in _plan(case) if r]
    tokens = sum(n for n, _ in rows)
    data = tokens * ((H + 2 * Hkv) * D * 2 + H * 4 + 4 + H * D * 2)  # qkv, gate, pos, out
    if op != "prefill_packed":
        data += tokens * 2 * Hkv * D * 2                             # the new keys and values
        data += sum(o - _first_key(case, o) for _, o in rows) * 2 * Hkv * D * 2
    flops = sum(_pairs(case, n, o) for n, o in rows) * H * D * 4
    return {"bytes": data, "flops": flops}


def _fork_rows(case):
    """Lengths of the parents, and (parent, child) pairs of row numbers."""
    p, n = case["parents"], case["copies"]
    return _spread(case["mix"], p, case["longest"]), [(i % p, p + i) for i in range(p * n)]


def _compact_rows(case):
    """Lengths of two groups of rows that take turns: even rows, odd rows."""
    half = case["rows"] // 2
    v = [0] * (2 * half)
    v[0::2] = _spread(case["mix"], half, case["longest"])
    v[1::2] = _spread(case["mix"] + 1, half, case["longest"])
    return v


def _page_work(case):
    """Pages that have to move in a pass, and the bytes of the tables."""
    page = case["page"]
    if case["op"] == "fork":
        lens, pairs = _fork_rows(case)
        moved = sum(case["copies"] for x in lens if x % page)
        held = sum(-(-x // page) for x in lens)
        return moved, 4 * held * (2 + 3 * case["copies"])
    need = [-(-x // page) for x in _compact_rows(case)]
    a, b = sum(need[0::2]), sum(need[1::2])
    return min(a, b), 4 * 3 * (a + b)   # either group's pages close the other's gap


# ---------------------------------------------------------------- inputs

def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _pool(g, *shape):
    """bf16 normal values, drawn layer by layer (or in one piece)."""
    t = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    for part in (t if len(shape) == 5 else [t]):
        part.normal_(generator=g)
    return t


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    rng = random.Random(seed)
    s = {"case": case}
    if case["op"] in ("fork", "compact"):
        _prepare_pool(case, s, g)
        return s
    rows = _plan(case)
    new = [r[0] if r else 0 for r in rows]
    old = [r[1] if r else 0 for r in rows]
    width = (case["H"] + 2 * case["Hkv"]) * D
    tokens = len(rows) if case["op"] == "decode_paged" else sum(new) + case["pad"]
    s["qkv"] = _randn(g, tokens, width)
    s["gate"] = _randn(g, tokens, case["H"], dtype=torch.float32)
    s["out"] = torch.zeros((tokens, case["H"] * D), dtype=torch.bfloat16, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    if case["op"] == "decode_paged":
        s["pos"] = torch.tensor([r[1] if r else -1 for r in rows], **i32)
    else:
        pos = [torch.arange(o, o + n) for n, o in zip(new, old)] + [torch.zeros(case["pad"])]
        s["pos"] = torch.cat(pos).to(**i32)
        s["lens"] = new
        s["cu"] = torch.tensor([0] + new).cumsum(0).to(**i32)
        s["start"] = torch.tensor(old, **i32)
    if case["op"] != "prefill_packed":
        page = case["page"]
        span = [(_first_key(case, o) // page, -(-(o + n) // page)) if n else (0, 0)
                for n, o in zip(new, old)]   # pages from the window's first to the last token's
        n_pages = sum(b - a for a, b in span) * 9 // 8 + 3
        ids = list(range(n_pages))
        rng.shuffle(ids)
        table = torch.full((len(rows), max(b for _, b in span) + 2), -1, dtype=torch.int32)
        for i, (a, b) in enumerate(span):
            table[i, a:b] = torch.tensor([ids.pop() for _ in range(b - a)], dtype=torch.int32)
        s["table"] = table.to(DEV)
        s["old"] = old
        s["k"] = _pool(g, n_pages, case["Hkv"], page, D)
        s["v"] = _pool(g, n_pages, case["Hkv"], page, D)
    return s


def _prepare_pool(case, s, g):
    page, i32 = case["page"], dict(dtype=torch.int32, device=DEV)
    if case["op"] == "fork":
        lens, pairs = _fork_rows(case)
        n_rows = len(lens) + len(pairs)
        lens = lens + [0] * len(pairs)
        n_pages = sum(-(-x // page) for x in lens) + 2 * n_rows + 2
        s["src"] = torch.tensor([a for a, _ in pairs], **i32)
        s["dst"] = torch.tensor([b for _, b in pairs], **i32)
        s["add"] = torch.ones(n_rows, **i32)
    else:
        lens = _compact_rows(case)
        n_rows = len(lens)
        n_pages = sum(-(-x // page) for x in lens) + 3
        s["groups"] = [torch.arange(k, n_rows, 2, **i32) for k in (0, 1)]
        s["adds"] = []
        for k in (0, 1):
            add = torch.zeros(n_rows, **i32)
            add[k::2] = torch.tensor(lens[k::2], **i32)
            s["adds"].append(add)
        s["turn"] = 0
    held = [-(-x // page) for x in lens]
    table = torch.full((n_rows, max(held) + 2), -1, dtype=torch.int32)
    n = 0
    order = range(n_rows) if case["op"] == "fork" else [*range(0, n_rows, 2), *range(1, n_rows, 2)]
    for i in order:
        table[i, :held[i]] = torch.arange(n, n + held[i], dtype=torch.int32)
        n += held[i]
    s["table"] = table.to(DEV)
    s["held"] = torch.tensor(held, **i32)
    s["len"] = torch.tensor(lens, **i32)
    s["refs"] = (torch.arange(n_pages, device=DEV) < n).to(torch.int32)
    s["k"] = _pool(g, case["layers"], n_pages, case["Hkv"], page, D)
    s["v"] = _pool(g, case["layers"], n_pages, case["Hkv"], page, D)


# ---------------------------------------------------------------- a pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _own_state(s):
    """What a user's program keeps between calls: the layer and a zeroed workspace."""
    import full_gqa_attention_gb300 as fga
    if "ws" not in s:
        c = s["case"]
        if c["op"] in ("fork", "compact"):
            s["pool"] = fga.PagePool(s["k"], s["v"], s["table"], s["held"], s["len"], s["refs"])
            need = fga.spark_attn_pages_workspace_size(s["pool"])
        else:
            theta, rot = KINDS[c["kind"]]
            s["layer"] = fga.layer_desc(int(c["kind"] == "sliding"), c["window"], theta, rot)
            n = s["qkv"].shape[0]
            if c["op"] == "decode_paged":
                need = fga.spark_attn_decode_paged_workspace_size(n, c["H"], c["Hkv"], s["layer"])
            else:
                size = (fga.spark_attn_prefill_packed_workspace_size
                        if c["op"] == "prefill_packed"
                        else fga.spark_attn_prefill_paged_workspace_size)
                need = size(n, len(s["lens"]), c["H"], c["Hkv"], s["layer"])
        s["ws"] = fga.new_workspace(need)
    return fga


def _own_packed(s):
    fga = _own_state(s)
    return fga.spark_attn_prefill_packed(s["qkv"], s["gate"], s["pos"], s["cu"], s["layer"],
                                         out=s["out"], workspace=s["ws"])


def _own_paged(s):
    fga = _own_state(s)
    fga.spark_attn_prefill_paged(s["qkv"], s["gate"], s["pos"], s["cu"], s["start"], s["k"],
                                 s["v"], s["table"], s["layer"], out=s["out"],
                                 workspace=s["ws"])
    return {"out": s["out"], "k": s["k"], "v": s["v"]}


def _own_decode(s):
    fga = _own_state(s)
    fga.spark_attn_decode_paged(s["qkv"], s["gate"], s["pos"], s["k"], s["v"], s["table"],
                                s["layer"], out=s["out"], workspace=s["ws"])
    return {"out": s["out"], "k": s["k"], "v": s["v"]}


def _pool_state(s):
    return {n: s[n] for n in ("k", "v", "table", "held", "len", "refs")}


def _own_fork(s):
    fga = _own_state(s)
    fga.spark_attn_pages_free(s["pool"], s["dst"], workspace=s["ws"])
    fga.spark_attn_pages_fork(s["pool"], s["src"], s["dst"], workspace=s["ws"])
    fga.spark_attn_pages_reserve(s["pool"], s["add"], workspace=s["ws"])
    return _pool_state(s)


def _own_compact(s):
    fga = _own_state(s)
    turn = s["turn"]
    s["turn"] = 1 - turn
    fga.spark_attn_pages_free(s["pool"], s["groups"][turn], workspace=s["ws"])
    fga.spark_attn_pages_compact(s["pool"], workspace=s["ws"])
    fga.spark_attn_pages_reserve(s["pool"], s["adds"][turn], workspace=s["ws"])
    s["len"] += s["adds"][turn]
    return _pool_state(s)


# ---------------------------------------------------------------- plain forms

def _rotate(x, pos, kind):
    """x [n, heads, 256] in 32 bits, the first rot dims turned at pos [n]; the angles of far
    positions in 64 bits."""
    theta, r = KINDS[kind]
    freq = theta ** (-torch.arange(0, r, 2, device=x.device, dtype=torch.float64) / r)
    a = pos.double()[:, None] * freq
    c, s = a.cos().float()[:, None], a.sin().float()[:, None]
    x1, x2 = x[..., :r // 2], x[..., r // 2:r]
    return torch.cat([x1 * c - x2 * s, x2 * c + x1 * s, x[..., r:]], dim=-1)


def _split(s):
    """q in 32 bits, rotated; k as a page holds it (rotated, bf16); v."""
    c = s["case"]
    x = s["qkv"].view(-1, c["H"] + 2 * c["Hkv"], D)
    H, Hkv = c["H"], c["Hkv"]
    q = _rotate(x[:, :H].float(), s["pos"], c["kind"])
    k = _rotate(x[:, H:H + Hkv].float(), s["pos"], c["kind"]).to(torch.bfloat16)
    return q, k, x[:, H + Hkv:]


def _attend(q, k, v, gate, at, first, window):
    """Attention of the queries q [n, H, D] at indices at.. over the keys k [m, Hkv, D] at
    indices first.., in 32 bits, gated."""
    n, H, _ = q.shape
    m, Hkv, _ = k.shape
    qs = q.view(n, Hkv, H // Hkv, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D)
    x = torch.matmul(qs, k.float().permute(1, 2, 0)) / 16
    i = torch.arange(at, at + n, device=q.device)[:, None]
    j = torch.arange(first, first + m, device=q.device)
    hidden = j > i
    if window:
        hidden = hidden | (i - j >= window)
    x = x.view(Hkv, H // Hkv, n, m).masked_fill_(hidden, -math.inf)
    x = torch.exp(x.sub_(x.amax(-1, keepdim=True)))
    o = torch.matmul(x.view(Hkv, -1, m), v.float().transpose(0, 1))
    o = o.view(H, n, D) / x.sum(-1).view(H, n, 1)
    return o.transpose(0, 1) / (1 + torch.exp(-gate))[..., None]


ROWS = 2048   # queries at a time: the scores of a long prompt do not fit otherwise


def _prompts(s, q, gate, keys_of):
    """The outputs of packed prompts; keys_of(i, first, end) gives sequence i's keys and values."""
    c = s["case"]
    window = c["window"] if c["kind"] == "sliding" else 0
    out = torch.zeros((q.shape[0], c["H"] * D), dtype=torch.bfloat16, device=q.device)
    t = 0
    olds = s.get("old", [0] * len(s["lens"]))
    for i, n in enumerate(s["lens"]):
        for a in range(0, n, ROWS):
            b, at = min(a + ROWS, n), olds[i] + a
            first = max(0, at - window + 1) if window else 0
            k, v = keys_of(i, t - olds[i], first, olds[i] + b)
            o = _attend(q[t + a:t + b], k, v, gate[t + a:t + b], at, first, window)
            out[t + a:t + b] = o.reshape(b - a, -1).to(torch.bfloat16)
        t += n
    return out


def _plain_packed(s):
    q, k, v = _split(s)
    return _prompts(s, q, s["gate"], lambda i, t, a, b: (k[t + a:t + b], v[t + a:t + b]))


def _plain_paged(s):
    c = s["case"]
    page = c["page"]
    q, k, v = _split(s)
    n = sum(s["lens"])
    seq = torch.repeat_interleave(torch.arange(len(s["lens"]), device=DEV),
                                  torch.tensor(s["lens"], device=DEV))
    at = s["pos"][:n].long()
    ids = s["table"][seq, at // page].long()
    s["k"][ids, :, at % page] = k[:n]
    s["v"][ids, :, at % page] = v[:n]

    def keys_of(i, t, a, b):
        p0 = a // page
        ids = s["table"][i, p0:-(-b // page)].long()
        return [x[ids].transpose(1, 2).reshape(-1, c["Hkv"], D)[a - p0 * page:b - p0 * page]
                for x in (s["k"], s["v"])]

    return {"out": _prompts(s, q, s["gate"], keys_of), "k": s["k"], "v": s["v"]}


def _plain_decode(s):
    c = s["case"]
    page, H, Hkv = c["page"], c["H"], c["Hkv"]
    q, k, v = _split(s)
    live = (s["pos"] >= 0).nonzero()[:, 0]
    pos = s["pos"][live].long()
    q, k, v, table = q[live], k[live], v[live], s["table"][live].long()
    ids = table.gather(1, (pos // page)[:, None])[:, 0]
    s["k"][ids, :, pos % page] = k
    s["v"][ids, :, pos % page] = v
    lo = (pos - c["window"] + 1).clamp(min=0) if c["kind"] == "sliding" else pos * 0
    p0 = lo // page
    most = int((pos // page - p0).max()) + 1
    cols = p0[:, None] + torch.arange(most, device=DEV)
    ids = table.gather(1, cols.clamp(max=table.shape[1] - 1)).clamp(min=0)
    j = cols[:, :, None] * page + torch.arange(page, device=DEV)
    seen = ((j >= lo[:, None, None]) & (j <= pos[:, None, None])).flatten(1)     # [B, m]
    K, V = (x[ids].transpose(1, 2).reshape(len(live), Hkv, -1, D).float()
            for x in (s["k"], s["v"]))
    x = torch.matmul(q.view(-1, Hkv, H // Hkv, D), K.transpose(2, 3)) / 16
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    x = torch.exp(x.sub_(x.amax(-1, keepdim=True)))
    o = torch.matmul(x, V) / x.sum(-1, keepdim=True)
    o = o.view(-1, H, D) / (1 + torch.exp(-s["gate"][live]))[..., None]
    out = torch.zeros((len(s["pos"]), H * D), dtype=torch.bfloat16, device=DEV)
    out[live] = o.reshape(-1, H * D).to(torch.bfloat16)
    return {"out": out, "k": s["k"], "v": s["v"]}


def _plain_free(s, rows):
    """Gives back every page of the rows."""
    rows = rows.long()
    n_pages = s["refs"].numel()
    ids = s["table"][rows]
    ids = torch.where(torch.arange(ids.shape[1], device=DEV) < s["held"][rows][:, None], ids,
                      n_pages).long().flatten()
    gone = torch.zeros(n_pages + 1, dtype=torch.int32, device=DEV)
    gone.index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))
    s["refs"] -= gone[:-1]
    s["table"][rows] = -1
    s["held"][rows] = 0
    s["len"][rows] = 0


def _plain_reserve(s, add):
    """Room for add[r] more tokens in every row: free pages from the lowest number up, rows in
    order, in each the copy of a shared page first.  Of the rows about to write into one shared
    page all copy it but the last."""
    page = s["case"]["page"]
    table, refs, held, length = s["table"], s["refs"], s["held"], s["len"]
    n_rows, max_pages = table.shape
    row = torch.arange(n_rows, device=DEV)
    grows = add > 0
    last = table[row, (length // page).clamp(max=max_pages - 1).long()]
    writes = grows & (length % page != 0)              # into a page that holds tokens already
    same = writes[:, None] & writes[None, :] & (last[:, None] == last[None, :])
    before = (same & (row[None, :] < row[:, None])).sum(1)
    copies = writes & (refs[last.clamp(min=0).long()] - before > 1)
    fresh = torch.where(grows, (-(-(length + add) // page) - held).clamp(min=0), 0)
    want = fresh + copies
    first = want.cumsum(0) - want
    free = (refs == 0).nonzero()[:, 0].to(torch.int32)
    # copies
    r = copies.nonzero()[:, 0]
    old, new = last[r].long(), free[first[r].long()]
    for x in (s["k"], s["v"]):
        x[:, new.long()] = x[:, old]
    table[r, (length[r] // page).long()] = new
    refs.index_add_(0, old, torch.full_like(new, -1))
    # fresh pages
    col = torch.arange(max_pages, device=DEV)
    at = col - held[:, None]
    gets = (at >= 0) & (at < fresh[:, None])
    pick = (first + copies)[:, None] + at
    table[gets] = free[pick[gets].long()]
    held += fresh.to(torch.int32)
    refs[free[:int(want.sum())].long()] = 1


def _plain_fork(s):
    _plain_free(s, s["dst"])
    page, src, dst = s["case"]["page"], s["src"].long(), s["dst"].long()
    n = -(-s["len"][src] // page)
    n_pages, cols = s["refs"].numel(), torch.arange(s["table"].shape[1], device=DEV)
    ids = torch.where(cols < n[:, None], s["table"][src], -1)
    s["table"][dst] = ids
    s["held"][dst] = n
    s["len"][dst] = s["len"][src]
    more = torch.zeros(n_pages + 1, dtype=torch.int32, device=DEV)
    more.index_add_(0, torch.where(ids < 0, n_pages, ids).long().flatten(),
                    torch.ones(ids.numel(), dtype=torch.int32, device=DEV))
    s["refs"] += more[:-1]
    _plain_reserve(s, s["add"])
    return _pool_state(s)


def _plain_compact(s):
    turn = s["turn"]
    s["turn"] = 1 - turn
    _plain_free(s, s["groups"][turn])
    live = s["refs"] > 0
    n = int(live.sum())
    holes = (~live[:n]).nonzero()[:, 0]
    movers = live[n:].nonzero()[:, 0] + n
    for x in (s["k"], s["v"]):
        x[:, holes] = x[:, movers]
    to = torch.arange(live.numel(), device=DEV, dtype=torch.int32)
    to[movers] = holes.to(torch.int32)
    s["refs"][holes] = s["refs"][movers]
    s["refs"][movers] = 0
    held = torch.arange(s["table"].shape[1], device=DEV) < s["held"][:, None]
    s["table"][held] = to[s["table"][held].long()]
    _plain_reserve(s, s["adds"][turn])
    s["len"] += s["adds"][turn]
    return _pool_state(s)


_OWN = {"prefill_packed": _own_packed, "prefill_paged": _own_paged, "decode_paged": _own_decode,
        "fork": _own_fork, "compact": _own_compact}
_PLAIN = {"prefill_packed": _plain_packed, "prefill_paged": _plain_paged,
          "decode_paged": _plain_decode, "fork": _plain_fork, "compact": _plain_compact}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("fork", "compact"):
        return _exact_pages(case, s)
    theta, rot = KINDS[case["kind"]]
    H, Hkv, G = case["H"], case["Hkv"], case["H"] // case["Hkv"]
    x = s["qkv"].double().view(-1, H + 2 * Hkv, D)
    angle = torch.outer(s["pos"].double(), torch.exp(
        -math.log(theta) * 2 / rot * torch.arange(rot // 2, device=DEV, dtype=torch.float64)))
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    z = torch.complex(x[:, :H + Hkv, :rot // 2], x[:, :H + Hkv, rot // 2:rot]) * turn
    x[:, :H + Hkv, :rot] = torch.cat([z.real, z.imag], dim=-1)
    key = x[:, H:H + Hkv].to(torch.bfloat16)
    value = s["qkv"].view(-1, H + 2 * Hkv, D)[:, H + Hkv:]
    out = torch.zeros((x.shape[0], H, D), dtype=torch.float64, device=DEV)
    t = 0
    for i, r in enumerate(_plan(case)):
        if r is None:
            t += case["op"] == "decode_paged"
            continue
        n, old = r
        if case["op"] == "prefill_packed":
            k, v, base = key[t:t + n], value[t:t + n], 0
        else:
            # the sequence's pages, from the first that anything is read of
            page = case["page"]
            p0 = _first_key(case, old) // page
            base = p0 * page
            ids = s["table"][i, p0:-(-(old + n) // page)].tolist()
            for j in range(old, old + n):
                s["k"][ids[j // page - p0], :, j % page] = key[t + j - old]
                s["v"][ids[j // page - p0], :, j % page] = value[t + j - old]
            k = torch.cat([s["k"][p].transpose(0, 1) for p in ids])
            v = torch.cat([s["v"][p].transpose(0, 1) for p in ids])
        for a in range(0, n, 1024):
            b = min(a + 1024, n)
            i0, end = old + a, old + b          # indices of these queries
            lo = max(0, i0 - case["window"] + 1) if case["kind"] == "sliding" else 0
            gap = (torch.arange(i0, end, device=DEV)[:, None]
                   - torch.arange(lo, end, device=DEV)[None, :])
            seen = gap >= 0
            if case["kind"] == "sliding":
                seen &= gap < case["window"]
            for h in range(H):
                kk = k[lo - base:end - base, h // G].double()
                w = x[t + a:t + b, h] @ kk.T * 0.0625
                w[~seen] = -math.inf
                w -= torch.logsumexp(w, dim=1, keepdim=True)
                out[t + a:t + b, h] = (w.exp_() @ v[lo - base:end - base, h // G].double()
                                       * torch.sigmoid(s["gate"][t + a:t + b, h:h + 1].double()))
        t += n
    out = out.view(-1, H * D)
    if case["op"] == "prefill_packed":
        return out
    return {"out": out, "k": s["k"], "v": s["v"]}


def _exact_pages(case, s):
    """The tables one step after another on the host, the pages copied as they say."""
    page = case["page"]
    table, held, length, refs = (s[n].tolist() for n in ("table", "held", "len", "refs"))

    def free(r):
        for p in table[r][:held[r]]:
            refs[p] -= 1
        table[r], held[r], length[r] = [-1] * len(table[r]), 0, 0

    def copy(p, q):
        s["k"][:, q] = s["k"][:, p]
        s["v"][:, q] = s["v"][:, p]

    def reserve(add):
        spare = [p for p, n in enumerate(refs) if n == 0]
        for r, more in enumerate(add):
            if not more:
                continue
            if length[r] % page:
                at = length[r] // page
                p = table[r][at]
                if refs[p] > 1:
                    q = table[r][at] = spare.pop(0)
                    refs[p], refs[q] = refs[p] - 1, 1
                    copy(p, q)
            while held[r] * page < length[r] + more:
                q = table[r][held[r]] = spare.pop(0)
                refs[q] = 1
                held[r] += 1

    if case["op"] == "fork":
        pairs = list(zip(s["src"].tolist(), s["dst"].tolist()))
        for _, d in pairs:
            free(d)
        for a, d in pairs:
            n = -(-length[a] // page)
            table[d][:n], held[d], length[d] = table[a][:n], n, length[a]
            for p in table[d][:n]:
                refs[p] += 1
        reserve(s["add"].tolist())
    else:
        for r in s["groups"][0].tolist():
            free(r)
        n = sum(x > 0 for x in refs)
        holes = [p for p in range(n) if refs[p] == 0]
        for p in range(n, len(refs)):
            if refs[p] > 0:
                q = holes.pop(0)
                copy(p, q)
                refs[q], refs[p] = refs[p], 0
                for r in range(len(table)):
                    table[r] = [q if x == p else x for x in table[r]]
        add = s["adds"][0].tolist()
        reserve(add)
        length = [a + b for a, b in zip(length, add)]
    back = {n: torch.tensor(v, dtype=torch.int32, device=DEV)
            for n, v in (("table", table), ("held", held), ("len", length), ("refs", refs))}
    return {"k": s["k"], "v": s["v"], **back}
