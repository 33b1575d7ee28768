"""pa_decode_scores and pa_evict on the GPU: decode that adds up attention weights, and
eviction by them, against 64-bit references; then a serving loop that uses both."""
import numpy as np
import pytest
import torch

from pa_ops_testlib import EPS32, Paged, attend, logit_error
from pa_testlib import TOL, bits, max_abs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_363_b200 import pa as _pa
    return _pa


def _scores_ref(p, q, scale, G):
    """out, weights summed over each kv head's heads, and the weights' error bound."""
    S, Hq, D = q.shape
    out = np.zeros((S, Hq, D))
    w, tol = {}, {}
    for s, L in enumerate(p.lens):
        for h in range(p.Hkv):
            k, v = p.rows(s, h)
            o, pr, _, mags = attend(q[s, h * G:(h + 1) * G].double().numpy(), k, v, scale)
            out[s, h * G:(h + 1) * G] = o
            w[s, h] = pr.sum(0)
            # a weight is 2^(x - M) / l: the logit's error counts for x, for M and for every term of l (3 times),
            # exp2f, the division, the products and the sum over heads are some 20 roundings more
            tol[s, h] = (pr * (3 * logit_error(mags, D).max(initial=0.0) + 32 * EPS32)).sum(0)
    return out, w, tol


@pytest.mark.parametrize("dt,Hkv,G,D,B,part", [
    ("bf16", 3, 1, 128, 16, 0), ("bf16", 2, 2, 64, 32, 64), ("bf16", 2, 4, 128, 16, 32), ("bf16", 1, 8, 64, 16, 0),
    ("f32", 2, 1, 64, 16, 0), ("f32", 1, 2, 128, 32, 32), ("f32", 2, 4, 64, 16, 512), ("f32", 1, 8, 128, 16, 48)])
def test_scores_against_the_definition(pa, dt, Hkv, G, D, B, part):
    tdt = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    lens = [1, 0, 2, 15, 16, 17, 100, 640, 1, 333]
    p = Paged(lens, Hkv, B, D, tdt, seed=G * D + B)
    q = p.q(len(lens), Hkv * G)
    k, v, tables, ctx = p.cuda()
    W = max(lens) + 5
    start = torch.rand(len(lens), Hkv, W, generator=torch.Generator().manual_seed(3)) * 4
    for s, L in enumerate(lens):
        if L:
            start[s, :, L - 1] = float("nan")        # what an earlier token left: the call sets this entry
    scores = start.cuda()
    out = torch.empty(q.shape, dtype=tdt, device="cuda")
    plain = torch.empty_like(out)
    scale = D ** -0.5
    pa.pa_decode_scores(out, scores, q.cuda(), k, v, tables, ctx, max(lens), scale, part)
    pa.pa_decode(plain, q.cuda(), k, v, tables, ctx, max(lens), scale, part)
    torch.cuda.synchronize()
    assert pa.pa_device_status() == 0
    ref, w, tol = _scores_ref(p, q, scale, G)
    assert np.array_equal(bits(out), bits(plain))     # the attention itself is pa_decode's
    assert max_abs(out.float().cpu().numpy(), ref) <= TOL[dt]
    got = scores.cpu().double().numpy()
    for s, L in enumerate(lens):
        for h in range(Hkv):
            if L:
                want = start[s, h, :L].double().numpy() + w[s, h]
                want[L - 1] = w[s, h][L - 1]
                assert np.all(np.abs(got[s, h, :L] - want) <= tol[s, h] + 2 * EPS32 * np.abs(want)), (s, h)
                assert abs(w[s, h].sum() - G) < 1e-9
            assert np.array_equal(got[s, h, L:], start[s, h, L:].double().numpy(), equal_nan=True)


def test_scores_same_bits_each_time_and_when_replayed(pa):
    lens = [700, 64, 1500, 9]
    p = Paged(lens, 2, 16, 128, torch.bfloat16, seed=4)
    q = p.q(4, 8).cuda()
    k, v, tables, ctx = p.cuda()
    ws = torch.empty(pa.pa_decode_scores_workspace_size(4, 8, 2, 128, 16, 1500), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)

    def call(sc, stream=None):
        pa.pa_decode_scores(out, sc, q, k, v, tables, ctx, 1500, 0.09, workspace=ws, stream=stream)
    a = torch.zeros(4, 2, 1500, device="cuda")
    b, c = a.clone(), a.clone()
    for _ in range(3):
        call(a)
    for _ in range(3):
        call(b)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        call(c, side)
    c.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, c)
    assert pa.pa_device_status() == 0


# ---------------------------------------------------------------- eviction

def _evict_ref(score, pos, n, recent):
    """Source slot of each of the first n slots."""
    L = len(score)
    if n >= L:
        return np.arange(min(n, L))
    safe = pos > pos.max() - min(recent, n)
    key = np.where(np.isnan(score), np.inf, score + 0.0)
    order = np.lexsort((np.arange(L), -key, ~np.isnan(score), ~safe))
    kept = np.zeros(L, bool)
    kept[order[:n]] = True
    src = np.arange(n)
    src[np.flatnonzero(~kept[:n])] = n + np.flatnonzero(kept[n:])
    return src


def _evict_case(lens, keep, Hkv, B, D, dt, seed, kind="random"):
    p = Paged(lens, Hkv, B, D, dt, seed)
    S, W = len(lens), max(max(lens), 1) + 3
    r = np.random.default_rng(seed + 1)
    sc = np.exp(r.standard_normal((S, Hkv, W)) * 2).astype(np.float32)
    if kind == "ties":
        sc = r.integers(0, 3, size=(S, Hkv, W)).astype(np.float32)
    elif kind == "odd":
        sc[r.random(sc.shape) < 0.1] = np.inf
        sc[r.random(sc.shape) < 0.1] = np.nan
        sc[r.random(sc.shape) < 0.2] = -0.0
        sc[r.random(sc.shape) < 0.2] = 0.0
        sc[r.random(sc.shape) < 0.1] = -1.5
        sc[r.random(sc.shape) < 0.1] = -np.inf
    pos = np.tile(np.arange(W, dtype=np.int32), (S, Hkv, 1))
    for s in range(0, S, 2):
        for h in range(Hkv):
            pos[s, h, :lens[s]] = r.permutation(lens[s]) + 1000
    return p, sc, pos, np.asarray(keep, np.int32)


def _run_evict(pa, p, sc, pos, keep, recent, alias):
    k, v, tables, ctx = p.cuda()
    a, b = torch.from_numpy(sc).cuda(), torch.from_numpy(pos).cuda()
    na, nb = (a, b) if alias else (torch.full_like(a, -7.0), torch.full_like(b, -7))
    pa.pa_evict(k, v, na, nb, a, b, tables, ctx, torch.from_numpy(keep).cuda(), recent, max(p.lens))
    torch.cuda.synchronize()
    return k.cpu(), v.cpu(), na.cpu().numpy(), nb.cpu().numpy()


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("dt,Hkv,D,B,kind,recent", [
    ("bf16", 2, 128, 16, "random", 8), ("bf16", 1, 64, 32, "ties", 0), ("f32", 3, 128, 32, "odd", 5),
    ("f32", 1, 64, 16, "random", 1000), ("bf16", 2, 128, 32, "odd", 0)])
def test_evict_bit_exact(pa, dt, Hkv, D, B, kind, recent, alias):
    tdt = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    lens = [1, 0, 31, 32, 33, 100, 257, 1025, 3000, 64, 5]
    keep = [1, 4, 30, 1, 32, 50, 256, 300, 2999, 64, 0]
    p, sc, pos, kp = _evict_case(lens, keep, Hkv, B, D, tdt, seed=D + B + recent, kind=kind)
    k, v, nsc, npos = _run_evict(pa, p, sc, pos, kp, recent, alias)
    assert pa.pa_device_status() == 0
    want_k, want_v = p.k.clone(), p.v.clone()
    for s, L in enumerate(lens):
        n = min(keep[s], L)
        for h in range(Hkv):
            src = _evict_ref(sc[s, h, :L].astype(np.float64), pos[s, h, :L], n, recent)
            assert np.array_equal(nsc[s, h, :n], sc[s, h, src], equal_nan=True), (s, h)
            assert np.array_equal(npos[s, h, :n], pos[s, h, src]), (s, h)
            i = np.arange(n)
            d, f = (p.tables[s][i // B], i % B), (p.tables[s][src // B], src % B)
            want_k[d[0], h, d[1]] = p.k[f[0], h, f[1]]
            want_v[d[0], h, d[1]] = p.v[f[0], h, f[1]]
            rest = sc[s, h, n:] if alias else np.full_like(sc[s, h, n:], -7.0)
            assert np.array_equal(nsc[s, h, n:], rest, equal_nan=True)
    assert np.array_equal(bits(k), bits(want_k)) and np.array_equal(bits(v), bits(want_v))


@pytest.mark.parametrize("dt,Hkv,D,B,recent", [("bf16", 8, 128, 16, 16), ("bf16", 8, 64, 32, 0), ("f32", 8, 128, 32, 33),
                                                ("f32", 16, 64, 16, 7)])
def test_evict_many_heads(pa, dt, Hkv, D, B, recent):
    """A kv head per SM and more: the rows are moved by the kernel that selects them."""
    tdt = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    rng = np.random.default_rng(D + B)
    lens = [1, 0, 4000, 33, 700] + rng.integers(1, 300, 18).tolist()
    keep = [1, 3, 100, 32, 699] + [int(rng.integers(0, L + 2)) for L in lens[5:]]
    p, sc, pos, kp = _evict_case(lens, keep, Hkv, B, D, tdt, seed=D + Hkv, kind="odd")
    assert len(lens) * Hkv >= 148
    for alias in (False, True):
        k, v, nsc, npos = _run_evict(pa, p, sc, pos, kp, recent, alias)
        assert pa.pa_device_status() == 0
        want_k, want_v = p.k.clone(), p.v.clone()
        for s, L in enumerate(lens):
            n = min(keep[s], L)
            for h in range(Hkv):
                src = _evict_ref(sc[s, h, :L].astype(np.float64), pos[s, h, :L], n, recent)
                assert np.array_equal(nsc[s, h, :n], sc[s, h, src], equal_nan=True), (s, h)
                assert np.array_equal(npos[s, h, :n], pos[s, h, src]), (s, h)
                i = np.arange(n)
                d, f = (p.tables[s][i // B], i % B), (p.tables[s][src // B], src % B)
                want_k[d[0], h, d[1]] = p.k[f[0], h, f[1]]
                want_v[d[0], h, d[1]] = p.v[f[0], h, f[1]]
        assert np.array_equal(bits(k), bits(want_k)) and np.array_equal(bits(v), bits(want_v))


def test_evict_bad_blocks_with_many_heads(pa):
    p, sc, pos, kp = _evict_case([100] * 24, [50] * 24, 8, 16, 64, torch.float32, seed=6)
    p.tables[3, :] = 10 ** 6
    p.tables[5, 6] = -1                                     # a block that only movers may lie in
    k, v, nsc, npos = _run_evict(pa, p, sc, pos, kp, 4, False)
    assert pa.pa_device_status() == pa.PA_DEV_BAD_BLOCK
    src = _evict_ref(sc[0, 0, :100].astype(np.float64), pos[0, 0, :100], 50, 4)
    i = np.arange(50)
    assert np.array_equal(bits(k[p.tables[0][i // 16], 0, i % 16]), bits(p.k[p.tables[0][src // 16], 0, src % 16]))


def test_evict_context_past_what_shared_memory_holds(pa):
    p, sc, pos, kp = _evict_case([60001, 9], [30000, 4], 1, 32, 64, torch.bfloat16, seed=19, kind="odd")
    k, v, nsc, npos = _run_evict(pa, p, sc, pos, kp, 77, False)
    assert pa.pa_device_status() == 0
    src = _evict_ref(sc[0, 0, :60001].astype(np.float64), pos[0, 0, :60001], 30000, 77)
    assert np.array_equal(npos[0, 0, :30000], pos[0, 0, src])


def test_evict_long_context(pa):
    lens, keep = [40000, 20001], [1000, 19000]
    p, sc, pos, kp = _evict_case(lens, keep, 1, 32, 64, torch.bfloat16, seed=9)
    k, v, nsc, npos = _run_evict(pa, p, sc, pos, kp, 100, False)
    assert pa.pa_device_status() == 0
    for s, L in enumerate(lens):
        src = _evict_ref(sc[s, 0, :L].astype(np.float64), pos[s, 0, :L], keep[s], 100)
        assert np.array_equal(npos[s, 0, :keep[s]], pos[s, 0, src])
        i = np.arange(keep[s])
        got = k[p.tables[s][i // 32], 0, i % 32]
        assert np.array_equal(bits(got), bits(p.k[p.tables[s][src // 32], 0, src % 32]))


def test_evict_flags_bad_lengths_and_blocks(pa):
    lens = [100, 90, 80]
    p, sc, pos, kp = _evict_case(lens, [50, -1, 40], 2, 16, 64, torch.float32, seed=5)
    p.tables[2, :] = 10 ** 6                                # blocks outside the pool: flagged, not touched
    k, v, nsc, npos = _run_evict(pa, p, sc, pos, kp, 4, False)
    assert pa.pa_device_status() == pa.PA_DEV_BAD_CONTEXT | pa.PA_DEV_BAD_BLOCK
    assert np.all(npos[1] == -7)
    src = _evict_ref(sc[0, 0, :100].astype(np.float64), pos[0, 0, :100], 50, 4)
    assert np.array_equal(npos[0, 0, :50], pos[0, 0, src])
    own = set(p.tables[0, :7].tolist())
    others = [b for b in range(p.k.shape[0]) if b not in own]
    assert np.array_equal(bits(k[others]), bits(p.k[others]))
    p.lens[0] = 10 ** 6                                     # a context past its table row
    k2, v2, tables, ctx = p.cuda()
    a, b = torch.from_numpy(sc).cuda(), torch.from_numpy(pos).cuda()
    pa.pa_evict(k2, v2, a.clone(), b.clone(), a, b, tables, ctx, torch.from_numpy(kp).cuda(), 4, 100)
    assert pa.pa_device_status() & pa.PA_DEV_BAD_CONTEXT


def test_decode_score_evict_loop(pa):
    """A serving loop: decode with scores, and back to the budget whenever it is exceeded, with one
    prompt forked into two streams.  Each step's attention is checked against the tokens that the
    reference's own bookkeeping says each head still holds."""
    Hkv, G, D, B, NB, budget, slack, recent = 2, 2, 64, 16, 64, 40, 6, 8
    W = budget + slack + 1
    rng = np.random.default_rng(0)
    a = pa.Allocator(NB, B)
    kc = torch.full((NB, Hkv, B, D), float("nan"), device="cuda")
    vc = kc.clone()
    put = lambda x, t: torch.from_numpy(np.ascontiguousarray(x, dtype=t)).cuda()  # noqa: E731
    prompt = 37
    slots = a.add_seq(0, prompt)
    kv = rng.standard_normal((2, prompt, Hkv, D)).astype(np.float32)
    pa.pa_reshape_and_cache(put(kv[0], np.float32), put(kv[1], np.float32), kc, vc, put(slots, np.int64))
    a.fork(0, 1)
    scores = torch.zeros(2, Hkv, W, device="cuda")
    positions = torch.arange(W, dtype=torch.int32, device="cuda").expand(2, Hkv, W).contiguous()
    held = [[[(i, kv[0, i, h], kv[1, i, h], 0.0) for i in range(prompt)] for h in range(Hkv)] for _ in range(2)]
    ids = np.array([0, 1])
    evicted = 0
    for step in range(24):
        slots, cow = a.append_slots(ids)
        if len(cow):
            pa.pa_copy_blocks(kc, vc, put(cow, np.int64))
        new = rng.standard_normal((2, 2, Hkv, D)).astype(np.float32)
        pa.pa_reshape_and_cache(put(new[0], np.float32), put(new[1], np.float32), kc, vc, put(slots, np.int64))
        tables, lens = a.block_tables(ids, 8)
        q = rng.standard_normal((2, Hkv * G, D)).astype(np.float32)
        out = torch.empty(2, Hkv * G, D, device="cuda")
        for s in range(2):
            positions[s, :, int(lens[s]) - 1] = prompt + step
        pa.pa_decode_scores(out, scores, put(q, np.float32), kc, vc, put(tables, np.int32), put(lens, np.int32), W, 0.3)
        got, sc = out.cpu().numpy(), scores.cpu().numpy()
        for s in range(2):
            for h in range(Hkv):
                held[s][h].append((prompt + step, new[0, s, h], new[1, s, h], 0.0))
                t = held[s][h]
                assert len(t) == lens[s]
                o, pr, _, _ = attend(q[s, h * G:(h + 1) * G], np.array([x[1] for x in t], np.float64),
                                     np.array([x[2] for x in t], np.float64), 0.3)
                assert max_abs(got[s, h * G:(h + 1) * G], o) <= TOL["f32"]
                held[s][h] = [(x[0], x[1], x[2], x[3] + w) for x, w in zip(t, pr.sum(0))]
                assert max_abs(sc[s, h, :len(t)], [x[3] for x in held[s][h]]) <= 1e-4
        if lens[0] > budget + slack - 1:
            pairs = np.concatenate([a.make_private(i, budget) for i in ids])
            if len(pairs):
                pa.pa_copy_blocks(kc, vc, put(pairs, np.int64), check=True)
            tables, lens = a.block_tables(ids, 8)
            pos = positions.cpu().numpy()
            pa.pa_evict(kc, vc, scores, positions, scores, positions, put(tables, np.int32), put(lens, np.int32),
                        put([budget, budget], np.int32), recent, W)
            for s in range(2):
                for h in range(Hkv):
                    # the scores as the device has them: a rounding may not decide what the reference keeps
                    src = _evict_ref(sc[s, h, :lens[s]].astype(np.float64), pos[s, h, :lens[s]], budget, recent)
                    held[s][h] = [held[s][h][i] for i in src]
                    assert positions[s, h, :budget].tolist() == [x[0] for x in held[s][h]]
                a.truncate(int(ids[s]), budget)
            evicted += 1
    assert evicted >= 2
    assert pa.pa_device_status() == 0
    assert a.stats()["tokens"] == sum(a.num_tokens(int(i)) for i in ids)
