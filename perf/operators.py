"""Serving operators over the paged KV cache, as they are measured: cases, inputs, the plain form and the work.

  shared   pa_decode_shared     decode attention of a batch whose sequences share leading blocks (a system prompt, the
                                streams of one prompt): the shared blocks are attended to once for all of them
  cross    pa_cross_attention   attention of packed query rows to an encoder's states kept in blocks, no causal mask
  scores   pa_decode_scores     decode attention that also adds every token's attention weight to its running score
  evict    pa_evict             drops the tokens of the lowest scores from each kv head and closes the gaps

Where `own` is false run() computes them with elementary torch operations in 32 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the smallest call: the four streams of one short prompt, latency alone
        dict(name="shared-streams-small", op="shared", dtype="bf16", hq=8, hkv=8, d=64, bs=16, groups=1, members_lo=4,
             members_hi=4, shared_lo=90, shared_hi=120, own_lo=1, own_hi=20, single=0, lens=1),
        # 8 system prompts with 16 requests each, grouped-query heads: the prefix cache's batch
        dict(name="shared-prompts-gqa", op="shared", dtype="bf16", hq=32, hkv=8, d=128, bs=16, groups=8, members_lo=16,
             members_hi=16, shared_lo=512, shared_hi=1536, own_lo=16, own_hi=256, single=0, lens=2),
        # parallel sampling: 32 prompts with four streams each, one query head per kv head
        dict(name="shared-streams-mha", op="shared", dtype="bf16", hq=32, hkv=32, d=128, bs=16, groups=32, members_lo=4,
             members_hi=4, shared_lo=256, shared_hi=1024, own_lo=1, own_hi=40, single=0, lens=3),
        # questions about long documents, beside requests that share nothing
        dict(name="shared-documents-long", op="shared", dtype="bf16", hq=32, hkv=8, d=128, bs=32, groups=3, members_lo=10,
             members_hi=70, shared_lo=16384, shared_hi=32768, own_lo=1, own_hi=700, single=5, lens=4),
        # one new token per sequence, against the encoder states of inputs of very different lengths
        dict(name="cross-token-mha", op="cross", dtype="bf16", hq=16, hkv=16, d=64, bs=16, seqs=24, rows_lo=1, rows_hi=1,
             enc_lo=33, enc_hi=1500, lens=5),
        # a few candidate tokens per sequence, ragged, some sequences without one
        dict(name="cross-few-gqa", op="cross", dtype="bf16", hq=32, hkv=8, d=128, bs=16, seqs=48, rows_lo=0, rows_hi=9,
             enc_lo=100, enc_hi=2500, lens=6),
        # the decoder's prompts or training targets against whole encoder outputs
        dict(name="cross-prompts-gqa", op="cross", dtype="bf16", hq=32, hkv=8, d=128, bs=16, seqs=16, rows_lo=200,
             rows_hi=700, enc_lo=1000, enc_hi=3000, lens=7),
        # the tiny fp32 batch
        dict(name="scores-tiny-f32", op="scores", dtype="f32", hq=4, hkv=4, d=64, bs=16, seqs=4, ctx_lo=1, ctx_hi=100,
             lens=8),
        # 128 requests of ordinary, uneven lengths, grouped-query heads
        dict(name="scores-gqa", op="scores", dtype="bf16", hq=32, hkv=8, d=128, bs=16, seqs=128, ctx_lo=16, ctx_hi=4096,
             lens=9),
        # long contexts, where eviction pays
        dict(name="scores-long", op="scores", dtype="bf16", hq=32, hkv=8, d=128, bs=32, seqs=8, ctx_lo=16384,
             ctx_hi=32768, lens=10),
        # a step of ordinary serving: a small batch brought back to its budget
        dict(name="evict-budget", op="evict", dtype="bf16", hkv=8, d=128, bs=16, seqs=32, ctx_lo=1025, ctx_hi=1400,
             keep=1024, recent=128, lens=11),
        # long prompts cut down to a fixed budget after prefill
        dict(name="evict-long", op="evict", dtype="bf16", hkv=8, d=128, bs=32, seqs=8, ctx_lo=16384, ctx_hi=32768,
             keep=8192, recent=512, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "shared", "cross", "cross", "scores", "evict"])
    d, bs = rng.choice([64, 128, 128]), rng.choice([16, 16, 32])
    hkv = rng.choice([1, 2, 4, 8, 8, 16])
    g = rng.choice([1, 2, 4, 4, 8])
    c = dict(op=op, dtype="bf16", hq=hkv * g, hkv=hkv, d=d, bs=bs, lens=rng.randrange(1 << 20))
    if op == "shared":
        members = _log(rng, 2, 40)
        c.update(groups=_log(rng, 1, 12), members_lo=2, members_hi=members, own_lo=1, own_hi=_log(rng, 2, 600),
                 single=rng.choice([0, 0, 3]))
        hi = _log(rng, 40, 12000)
        c.update(shared_lo=max(bs, hi // 3), shared_hi=hi)
    elif op == "cross":
        rows, enc = _log(rng, 1, 500), _log(rng, 20, 3001)
        c.update(seqs=_log(rng, 1, 16), rows_lo=max(1, rows // 3), rows_hi=rows, enc_lo=max(1, enc // 4), enc_hi=enc)
    elif op == "scores":
        hi = _log(rng, 30, 20000)
        c.update(dtype=rng.choice(["bf16", "bf16", "f32"]), ctx_lo=max(1, hi // 5), ctx_hi=hi,
                 seqs=max(1, min(_log(rng, 1, 64), 100000 // hi)))
    else:
        hi = _log(rng, 100, 20000)
        keep = max(8, int(hi * rng.uniform(0.2, 0.9)))
        c.update(dtype=rng.choice(["bf16", "f32"]), ctx_lo=max(1, hi // 2), ctx_hi=hi, keep=keep,
                 recent=rng.randrange(keep // 2 + 1), seqs=max(1, min(_log(rng, 1, 48), 100000 // hi)))
        del c["hq"]
    return c


# ---------------------------------------------------------------- shapes (from the case alone)

def _shape(case):
    """The case's lengths: what its work is counted from and its inputs are made for."""
    rng = np.random.default_rng([20, case["lens"]])
    op, B = case["op"], case["bs"]
    z = {}
    if op == "shared":
        members = rng.integers(case["members_lo"], case["members_hi"] + 1, size=case["groups"])
        shared = rng.integers(case["shared_lo"], case["shared_hi"] + 1, size=case["groups"]) // B * B
        n = int(members.sum()) + case["single"]
        group = np.concatenate([np.repeat(np.arange(case["groups"]), members), np.full(case["single"], -1)])
        group = group[rng.permutation(n)]                # a batch's rows come in any order
        owned = rng.integers(case["own_lo"], case["own_hi"] + 1, size=n)
        z.update(group=group, shared=shared, ctx=np.where(group >= 0, shared[np.maximum(group, 0)], 0) + owned)
    elif op == "cross":
        rows = rng.integers(case["rows_lo"], case["rows_hi"] + 1, size=case["seqs"])
        rows[rng.integers(case["seqs"])] = case["rows_hi"]
        z.update(rows=rows, ctx=rng.integers(case["enc_lo"], case["enc_hi"] + 1, size=case["seqs"]))
    elif op == "scores":
        lo, hi = case["ctx_lo"], case["ctx_hi"]
        z["ctx"] = np.exp(rng.uniform(math.log(lo), math.log(hi), size=case["seqs"])).round().astype(np.int64)
    else:
        z["ctx"] = rng.integers(case["ctx_lo"], case["ctx_hi"] + 1, size=case["seqs"])
    return z


def _blocks(case, z):
    """Distinct blocks, and every sequence's own ones."""
    B = case["bs"]
    lead = np.zeros(len(z["ctx"]), np.int64)
    total = 0
    if case["op"] == "shared":
        lead = np.where(z["group"] >= 0, z["shared"][np.maximum(z["group"], 0)] // B, 0)
        total = int(sum(s // B for s in z["shared"]))
    each = -(-z["ctx"] // B) - lead
    return lead, each, total + int(each.sum())


def work(case):
    z = _shape(case)
    elt = 2 if case["dtype"] == "bf16" else 4
    Hkv, D, B = case["hkv"], case["d"], case["bs"]
    row = Hkv * D * elt * 2                                # K and V of one token
    ctx = z["ctx"]
    if case["op"] == "evict":
        keep = np.minimum(ctx, case["keep"])
        recent = np.minimum(case["recent"], keep)
        # tokens kept behind the budget, which move into the gaps before it: with tokens in order of age, and in any order
        heavy = np.where(ctx > keep, (keep - recent) * keep / np.maximum(np.maximum(ctx - recent, keep), 1), keep)
        moves = np.where(ctx > keep, ((keep - heavy) + keep * (1 - keep / np.maximum(ctx, 1))) / 2, 0)
        return {"bytes": float(Hkv * (8 * ctx + 8 * keep).sum() + 2 * row * moves.sum()), "flops": 0.0}
    Hq = case["hq"]
    lead, each, _ = _blocks(case, z)
    tables = 4 * int((-(-ctx // B)).sum() + len(ctx))
    rows = z.get("rows", np.ones(len(ctx), np.int64))
    tokens = int(ctx[rows > 0].sum()) if case["op"] == "cross" else int((ctx - lead * B).sum() + z.get("shared", np.zeros(1, int)).sum())
    nbytes = tokens * row + 2 * int(rows.sum()) * Hq * D * elt + tables
    if case["op"] == "scores":
        nbytes += 2 * 4 * Hkv * int(ctx.sum())
    return {"bytes": float(nbytes), "flops": float(4 * D * Hq * (rows * ctx).sum())}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    z = _shape(case)
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 9176 + 11)
    rng = np.random.default_rng([int(seed), 7])
    dt, Hkv, D, B = DTYPES[case["dtype"]], case["hkv"], case["d"], case["bs"]
    S = len(z["ctx"])
    lead, each, used = _blocks(case, z)
    NB = used + 3
    pool = torch.empty(2, NB, Hkv, B, D, dtype=dt, device=dev)
    for i in range(2):
        for b in range(0, NB, 4096):
            e = min(NB, b + 4096)
            pool[i, b:e] = torch.randn(e - b, Hkv, B, D, generator=g, device=dev).to(dt)
    # blocks lie anywhere in the pool, as an allocator leaves them
    perm = rng.permutation(NB)
    width = int((lead + each).max()) + 1
    tables = np.full((S, width), -1, np.int32)
    at = 0
    if case["op"] == "shared":
        starts = []
        for n in z["shared"] // B:
            starts.append(perm[at:at + n])
            at += int(n)
    for s in range(S):
        if lead[s]:
            tables[s, :lead[s]] = starts[z["group"][s]]
        tables[s, lead[s]:lead[s] + each[s]] = perm[at:at + each[s]]
        at += int(each[s])
    put = lambda a, t=np.int32: torch.from_numpy(np.ascontiguousarray(a, dtype=t)).to(dev)  # noqa: E731
    st = dict(op=case["op"], k=pool[0], v=pool[1], tables=put(tables), ctx=put(z["ctx"]), max_ctx=int(z["ctx"].max()),
              scale=1.0 / math.sqrt(D), lens=[int(x) for x in z["ctx"]])
    if case["op"] != "evict":
        n = int(z["rows"].sum()) if case["op"] == "cross" else S
        st["q"] = torch.randn(n, case["hq"], D, generator=g, device=dev).to(dt)
        st["out"] = torch.empty_like(st["q"])
    if case["op"] == "shared":
        rows = [np.flatnonzero(z["group"] == i) for i in range(case["groups"])]
        st.update(group_rows=put(np.concatenate(rows)), group_start=put(np.cumsum([0] + [len(r) for r in rows])),
                  shared_lens=put(z["shared"]), max_shared=int(z["shared"].max()),
                  members=[[int(x) for x in r] for r in rows], shared=[int(x) for x in z["shared"]])
    elif case["op"] == "cross":
        start = np.concatenate([[0], np.cumsum(z["rows"])])
        st.update(q_start=put(start), start=[int(x) for x in start], max_rows=int(z["rows"].max()),
                  lse=torch.empty(n, case["hq"], dtype=torch.float32, device=dev))
    elif case["op"] == "scores":
        # what earlier steps gave: a few tokens hold most of the weight
        st["scores"] = torch.randn(S, Hkv, st["max_ctx"], generator=g, device=dev).mul_(2).exp_()
    else:
        W = st["max_ctx"]
        sc = torch.randn(S, Hkv, W, generator=g, device=dev).mul_(2).exp_()
        sc[torch.rand(S, Hkv, W, generator=g, device=dev) < 0.05] = 0.0       # never attended to: ties
        pos = torch.arange(W, device=dev, dtype=torch.int32).expand(S, Hkv, W).clone()
        for s in range(1, S, 2):                                             # after earlier evictions: any order
            L = st["lens"][s]
            pos[s, :, :L] = torch.rand(Hkv, L, generator=g, device=dev).argsort(-1).to(torch.int32)
        keep = np.minimum(z["ctx"], case["keep"])
        st.update(scores=sc, positions=pos, keep_lens=put(keep), keep=[int(x) for x in keep], recent=case["recent"],
                  new_scores=torch.zeros_like(sc), new_positions=torch.zeros_like(pos))
    if own:
        from paged_kv_cache_363_b200 import pa
        Hq = case.get("hq", Hkv)
        if case["op"] == "shared":
            need = pa.pa_decode_shared_workspace_size(S, Hq, Hkv, D, B, st["max_ctx"], st["max_shared"], case["groups"],
                                                      int(st["group_rows"].numel()))
        elif case["op"] == "cross":
            need = pa.pa_cross_attention_workspace_size(S, Hq, Hkv, D, B, n, st["max_rows"], st["max_ctx"])
        elif case["op"] == "scores":
            need = pa.pa_decode_scores_workspace_size(S, Hq, Hkv, D, B, st["max_ctx"])
        else:
            need = pa.pa_evict_workspace_size(S, Hkv, st["max_ctx"])
        st["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    if own:
        return _run_own(st)
    return {"shared": _plain_shared, "cross": _plain_cross, "scores": _plain_scores, "evict": _plain_evict}[st["op"]](st)


def _run_own(st):
    from paged_kv_cache_363_b200 import pa
    if st["op"] == "shared":
        pa.pa_decode_shared(st["out"], st["q"], st["k"], st["v"], st["tables"], st["ctx"], st["group_rows"],
                            st["group_start"], st["shared_lens"], st["max_ctx"], st["max_shared"], st["scale"],
                            workspace=st["ws"])
        return [st["out"]]
    if st["op"] == "cross":
        pa.pa_cross_attention(st["out"], st["q"], st["k"], st["v"], st["tables"], st["ctx"], st["q_start"],
                              st["max_rows"], st["max_ctx"], st["scale"], lse=st["lse"], workspace=st["ws"])
        return [st["out"], st["lse"]]
    if st["op"] == "scores":
        pa.pa_decode_scores(st["out"], st["scores"], st["q"], st["k"], st["v"], st["tables"], st["ctx"], st["max_ctx"],
                            st["scale"], workspace=st["ws"])
        return [st["out"], st["scores"]]
    pa.pa_evict(st["k"], st["v"], st["new_scores"], st["new_positions"], st["scores"], st["positions"], st["tables"],
                st["ctx"], st["keep_lens"], st["recent"], st["max_ctx"], workspace=st["ws"])
    return [st["k"], st["v"], st["new_scores"], st["new_positions"]]


def _rows(pool, table, lo, hi):
    """Tokens lo .. hi-1 of one sequence, [Hkv, tokens, D] in 32 bits."""
    B = pool.shape[2]
    x = pool[table[lo // B:-(-hi // B)].long()].float()                     # [blocks, Hkv, B, D]
    return x.transpose(0, 1).reshape(pool.shape[1], -1, pool.shape[3])[:, lo % B:lo % B + hi - lo]


def _weights(q, k, scale):
    """q [rows, Hq, D], k [Hkv, tokens, D]: logits [Hkv, rows * G, tokens], their row maxima, exponentials and sums."""
    n, Hq, D = q.shape
    Hkv = k.shape[0]
    x = q.float().reshape(n, Hkv, Hq // Hkv, D).permute(1, 0, 2, 3).reshape(Hkv, -1, D)
    s = torch.matmul(x, k.transpose(1, 2)) * scale
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    return m, p, p.sum(-1, keepdim=True)


def _unpack(o, n):
    """[Hkv, n * G, X] back to [n, Hq, X]."""
    Hkv = o.shape[0]
    return o.reshape(Hkv, n, -1, o.shape[-1]).permute(1, 0, 2, 3).reshape(n, -1, o.shape[-1])


def _plain_shared(st):
    """The shared tokens once for all of a group's rows, each row's own tokens, and both joined."""
    out, scale = st["out"], st["scale"]
    lead = {}
    for rows, n in zip(st["members"], st["shared"]):
        if n == 0 or not rows:
            continue
        at = torch.tensor(rows, device=out.device)
        t = st["tables"][rows[0]]
        m, p, l = _weights(st["q"][at], _rows(st["k"], t, 0, n), scale)
        o = torch.matmul(p, _rows(st["v"], t, 0, n))
        m, l, o = (_unpack(x, len(rows)) for x in (m, l, o))
        for i, s in enumerate(rows):
            lead[s] = (n, m[i], l[i], o[i])
    for s, L in enumerate(st["lens"]):
        n, m0, l0, o0 = lead.get(s, (0, None, None, None))
        if L > n:
            t = st["tables"][s]
            m, p, l = _weights(st["q"][s:s + 1], _rows(st["k"], t, n, L), scale)
            o = torch.matmul(p, _rows(st["v"], t, n, L))
            m, l, o = (_unpack(x, 1)[0] for x in (m, l, o))
            if n:
                top = torch.maximum(m, m0)
                a, b = torch.exp(m - top), torch.exp(m0 - top)
                l, o = l * a + l0 * b, o * a + o0 * b
        else:
            l, o = l0, o0
        out[s] = (o / l).to(out.dtype)
    return [out]


def _plain_cross(st):
    out, lse = st["out"], st["lse"]
    for s, L in enumerate(st["lens"]):
        a, b = st["start"][s], st["start"][s + 1]
        if b > a:
            t = st["tables"][s]
            m, p, l = _weights(st["q"][a:b], _rows(st["k"], t, 0, L), st["scale"])
            o = torch.matmul(p, _rows(st["v"], t, 0, L)) / l
            out[a:b] = _unpack(o, b - a).to(out.dtype)
            lse[a:b] = _unpack(m + torch.log(l), b - a)[..., 0]
    return [out, lse]


def _plain_scores(st):
    out, scores = st["out"], st["scores"]
    for s, L in enumerate(st["lens"]):
        t = st["tables"][s]
        m, p, l = _weights(st["q"][s:s + 1], _rows(st["k"], t, 0, L), st["scale"])
        out[s] = _unpack(torch.matmul(p, _rows(st["v"], t, 0, L)) / l, 1)[0].to(out.dtype)
        w = (p / l).sum(1)                                  # over the group's query heads
        scores[s, :, :L - 1] += w[:, :L - 1]
        scores[s, :, L - 1] = w[:, L - 1]                   # the step's own token has no history
    return [out, scores]


def _plain_evict(st):
    k, v, B = st["k"], st["v"], st["k"].shape[2]
    dev, Hkv = k.device, k.shape[1]
    for s, L in enumerate(st["lens"]):
        n = st["keep"][s]
        sc, pos = st["scores"][s, :, :L], st["positions"][s, :, :L]
        if n < L:
            w = min(st["recent"], n)
            key = torch.where(pos > pos.amax(1, keepdim=True) - w, torch.full_like(sc, float("inf")), sc)
            order = torch.sort(key, dim=1, descending=True, stable=True).indices
            kept = torch.zeros(Hkv, L, dtype=torch.bool, device=dev)
            kept.scatter_(1, order[:, :n], True)
        else:
            kept = torch.ones(Hkv, L, dtype=torch.bool, device=dev)
        src = torch.arange(n, device=dev).repeat(Hkv, 1)
        hole = (~kept[:, :n]).nonzero()
        tail = kept[:, n:].nonzero()                        # as many, head by head, both in order
        src[hole[:, 0], hole[:, 1]] = tail[:, 1] + n
        st["new_scores"][s, :, :n] = sc.gather(1, src)
        st["new_positions"][s, :, :n] = pos.gather(1, src)
        t = st["tables"][s].long()
        h, d, f = hole[:, 0], hole[:, 1], tail[:, 1] + n
        for pool in (k, v):
            pool[t[d // B], h, d % B] = pool[t[f // B], h, f % B]
    return [k, v, st["new_scores"], st["new_positions"]]


# ---------------------------------------------------------------- the same in 64 bits, from the definitions

def exact(case, seed):
    global own
    mine, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = mine
    B, lens = case["bs"], st["lens"]
    if case["op"] == "evict":
        return _exact_evict(case, st)
    group = case["hq"] // case["hkv"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    lse = torch.zeros(out.shape[:2], dtype=torch.float64, device=out.device)
    scores = st["scores"].double() if case["op"] == "scores" else None
    for s, L in enumerate(lens):
        a, b = (st["start"][s], st["start"][s + 1]) if case["op"] == "cross" else (s, s + 1)
        i = torch.arange(L, device=out.device)
        blk, off = st["tables"][s].long()[i // B], i % B
        for h in range(case["hkv"]):
            kk, vv = st["k"][blk, h, off].double(), st["v"][blk, h, off].double()        # [L, D]
            heads = slice(h * group, (h + 1) * group)
            z = torch.einsum("ngd,ld->ngl", st["q"][a:b, heads].double(), kk) * st["scale"]
            lse[a:b, heads] = torch.logsumexp(z, -1)
            w = torch.softmax(z, -1)
            out[a:b, heads] = torch.einsum("ngl,ld->ngd", w, vv)
            if scores is not None:
                add = w[0].sum(0)
                scores[s, h, :L] += add
                scores[s, h, L - 1] = add[-1]
    return {"shared": [out], "cross": [out, lse], "scores": [out, scores]}[case["op"]]


def _exact_evict(case, st):
    B, Hkv = case["bs"], case["hkv"]
    sc, pos = st["scores"].double().cpu().numpy(), st["positions"].cpu().numpy()
    new_sc, new_pos = np.zeros_like(sc), np.zeros_like(pos)
    moves = []
    for s, L in enumerate(st["lens"]):
        n, table = st["keep"][s], st["tables"][s].cpu().numpy()
        for h in range(Hkv):
            x, y = sc[s, h, :L], pos[s, h, :L]
            safe = y > y.max() - min(st["recent"], n)
            order = np.lexsort((np.arange(L), -x, ~safe))   # the recent ones, then by score, then by place
            kept = np.zeros(L, bool)
            kept[order[:n]] = True
            src = np.arange(n)
            holes = np.flatnonzero(~kept[:n])
            src[holes] = n + np.flatnonzero(kept[n:])
            new_sc[s, h, :n], new_pos[s, h, :n] = x[src], y[src]
            f = src[holes]
            moves.append(np.stack([table[holes // B], np.full(len(f), h), holes % B, table[f // B], f % B]))
    m = torch.from_numpy(np.concatenate(moves, 1).astype(np.int64)).to(st["k"].device)
    pools = []
    for pool in (st["k"], st["v"]):
        pool[m[0], m[1], m[2]] = pool[m[3], m[1], m[4]]
        pools.append(pool.double())
    return pools + [torch.from_numpy(new_sc), torch.from_numpy(new_pos)]
