"""The serving operators where the other tests do not go: blocks past 2^31 elements of a pool, two streams at once, graphs
replayed with other lengths, score distributions that take the selection through all its passes, extremes of groups."""
import numpy as np
import pytest
import torch

from pa_ops_testlib import Paged
from test_gpu_scores_evict import _evict_ref, _run_evict
from test_gpu_shared import _batch, _call as shared_call, _check as shared_check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_363_b200 import pa as _pa
    return _pa


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def _ops(pa, k, v, tables, ctx, q, groups, lens, scores, stream=None, ws=(None,) * 6):
    """Every attention operator over one batch (q: [S, Hq, D], and four rows of it per sequence)."""
    rows, starts, shared = groups
    S, mx = q.shape[0], max(lens)
    G = q.shape[1] // k.shape[1]
    four = q.repeat_interleave(4, 0)
    many = q.repeat_interleave(256 // G, 0)
    outs = [torch.full_like(q, 7.0), torch.full_like(q, 7.0), torch.full_like(four, 7.0), torch.full_like(many, 7.0),
            torch.full_like(q, 7.0)]
    sc = scores.clone()
    pa.pa_decode_shared(outs[0], q, k, v, tables, ctx, rows, starts, shared, mx, int(max(shared.tolist() + [0])), 0.1,
                        workspace=ws[0], stream=stream)
    for o, x, n, w in ((outs[1], q, 1, ws[1]), (outs[2], four, 4, ws[2]), (outs[3], many, 256 // G, ws[3])):
        pa.pa_cross_attention(o, x, k, v, tables, ctx, _i32(np.arange(S + 1) * n), n, mx, 0.1, workspace=w, stream=stream)
    pa.pa_decode_scores(outs[4], sc, q, k, v, tables, ctx, mx, 0.1, workspace=ws[4], stream=stream)
    return outs + [sc]


def test_blocks_past_32_bits(pa):
    """The same blocks at the far end of pools of 2.4e9 elements each, bit for bit."""
    Hkv, G, D, B = 8, 4, 128, 16
    p, q, groups = _batch(Hkv, G, D, B, seed=40, groups=[(6, 15, [1, 40]), (3, 3, [200])], singles=[0, 700, 1])
    listed = (_i32(sum([g for g, _ in groups], [])), _i32(np.cumsum([0] + [len(g) for g, _ in groups])),
              _i32([n for _, n in groups]))
    k, v, tables, ctx = p.cuda()
    NB = k.shape[0]
    big = 148000
    scores = torch.rand(len(p.lens), Hkv, max(p.lens), device="cuda")
    near = _ops(pa, k, v, tables, ctx, q.cuda(), listed, p.lens, scores)
    K = torch.full((big, Hkv, B, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    V = torch.full_like(K, float("nan"))
    K[big - NB:], V[big - NB:] = k, v
    assert K.numel() > 2 ** 31
    moved = torch.where(tables >= 0, tables + (big - NB), tables)
    far = _ops(pa, K, V, moved, ctx, q.cuda(), listed, p.lens, scores)
    assert pa.pa_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(near, far))
    # eviction of the sequences that share nothing
    alone = [i for i in range(len(p.lens)) if i not in sum([g for g, _ in groups], [])]
    S, W = len(alone), max(p.lens)
    sc = torch.rand(S, Hkv, W, device="cuda")
    pos = torch.arange(W, dtype=torch.int32, device="cuda").expand(S, Hkv, W).contiguous()
    for kk, vv, tt in ((k, v, tables), (K, V, moved)):
        pa.pa_evict(kk, vv, sc.clone(), pos.clone(), sc, pos, tt[alone].contiguous(), ctx[alone].contiguous(),
                    _i32([50] * S), 8, W)
    torch.cuda.synchronize()
    assert pa.pa_device_status() == 0
    assert torch.equal(K[big - NB:].view(torch.int16), k.view(torch.int16))
    assert torch.equal(V[big - NB:].view(torch.int16), v.view(torch.int16))


def test_two_streams_at_once(pa):
    Hkv, G, D, B = 4, 4, 128, 16
    p, q, groups = _batch(Hkv, G, D, B, seed=41, groups=[(9, 60, [1, 40]), (3, 3, [200])], singles=[0, 2000, 1])
    listed = (_i32(sum([g for g, _ in groups], [])), _i32(np.cumsum([0] + [len(g) for g, _ in groups])),
              _i32([n for _, n in groups]))
    k, v, tables, ctx = p.cuda()
    qs = [q.cuda(), (q.float() * 0.5).to(torch.bfloat16).cuda()]
    scores = torch.rand(len(p.lens), Hkv, max(p.lens), device="cuda")
    want = [_ops(pa, k, v, tables, ctx, x, listed, p.lens, scores) for x in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(_ops(pa, k, v, tables, ctx, qs[i], listed, p.lens, scores, stream=s))
    torch.cuda.synchronize()
    assert pa.pa_device_status() == 0
    for i in range(2):
        for run in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(run, want[i]))


def test_replayed_with_other_lengths(pa):
    """A graph captured once serves any lengths below its bounds: everything about them is read on the device."""
    Hkv, G, D, B = 2, 4, 128, 16
    p, q, groups = _batch(Hkv, G, D, B, seed=42, groups=[(9, 30, [60, 100]), (4, 12, [300])], singles=[900, 1500, 64])
    S, mx = len(p.lens), max(p.lens)
    k, v, tables, ctx = p.cuda()
    qd = q.cuda()
    rows, starts, shared = (_i32(sum([g for g, _ in groups], [])), _i32(np.cumsum([0] + [len(g) for g, _ in groups])),
                            _i32([n for _, n in groups]))
    most = int(shared.max())
    qstart = _i32(np.arange(S + 1))
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (
        pa.pa_decode_shared_workspace_size(S, Hkv * G, Hkv, D, B, mx, most, 2, rows.numel()),
        pa.pa_cross_attention_workspace_size(S, Hkv * G, Hkv, D, B, S, 1, mx),
        pa.pa_cross_attention_workspace_size(S, Hkv * G, Hkv, D, B, S, 5, mx),
        pa.pa_decode_scores_workspace_size(S, Hkv * G, Hkv, D, B, mx))]
    scores = torch.zeros(S, Hkv, mx, device="cuda")

    def run(o, sc, stream=None):
        pa.pa_decode_shared(o[0], qd, k, v, tables, ctx, rows, starts, shared, mx, most, 0.1, workspace=ws[0], stream=stream)
        pa.pa_cross_attention(o[1], qd, k, v, tables, ctx, qstart, 1, mx, 0.1, workspace=ws[1], stream=stream)
        pa.pa_cross_attention(o[2], qd, k, v, tables, ctx, qstart, 5, mx, 0.1, workspace=ws[2], stream=stream)
        pa.pa_decode_scores(o[3], sc, qd, k, v, tables, ctx, mx, 0.1, workspace=ws[3], stream=stream)

    outs = [torch.empty_like(qd) for _ in range(4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        run(outs, scores, side)
    full = ctx.clone()
    cases = [(full, shared.clone(), qstart.clone()),
             (torch.clamp(full, max=500), torch.clamp(shared, max=320), qstart.clone()),
             (torch.clamp(full, max=33), _i32([32, 0]), _i32([0] * 3 + list(range(S - 2)))),  # three sequences without a row
             (torch.zeros_like(full), _i32([0, 0]), qstart.clone())]
    for c, n, st in cases:
        ctx.copy_(c)
        shared.copy_(n)
        qstart.copy_(st)
        for o in outs:
            o.fill_(7.0)
        scores.fill_(1.0)
        g.replay()
        torch.cuda.synchronize()
        again, sc = [torch.full_like(o, 7.0) for o in outs], torch.ones_like(scores)
        run(again, sc)
        torch.cuda.synchronize()
        assert pa.pa_device_status() == 0
        assert all(torch.equal(a, b) for a, b in zip(outs, again)) and torch.equal(scores, sc)
        p.lens = [int(x) for x in c]
        shared_check(p, q, outs[0], 0.1, G)


@pytest.mark.parametrize("kind", ["equal", "ties", "odd", "spread", "crowd", "recent"])
@pytest.mark.parametrize("count", [2, 5, 6])
def test_evict_selection(pa, kind, count):
    """Contexts of every kind of storage, and scores that end the selection in its first pass, its last, or on equals."""
    lens = [300, 4096, 4097, 9000, 30000, 50000][:count]
    keep = [129, 2000, 4000, 1, 29999, 20011][:count]
    p = Paged(lens, 1, 16, 64, torch.bfloat16, seed=50)
    r = np.random.default_rng(51)
    S, W = len(lens), max(lens)
    sc = np.exp(3 * r.standard_normal((S, 1, W))).astype(np.float32)
    pos = np.stack([r.permutation(W).astype(np.int32)[None] for _ in lens])
    for s, L in enumerate(lens):
        pos[s, 0, :L] = r.permutation(L)
    recent = 64
    if kind == "equal":
        sc[:] = 0.25
    elif kind == "ties":
        sc = r.integers(0, 5, sc.shape).astype(np.float32)
    elif kind == "odd":
        for x in (np.inf, -np.inf, np.nan, 0.0, -0.0, -2.5, 1e-42):
            sc[r.random(sc.shape) < 0.12] = x
        recent = 0
    elif kind == "spread":                                # outliers leave nearly all keys in one bin
        sc = (1.0 + r.random(sc.shape) * 1e-4).astype(np.float32)
        sc[:, :, 5], sc[:, :, 17] = 3e38, -3e38
    elif kind == "crowd":                                 # bins of more than 256 neighbours
        sc = (np.float32(1.0) + r.integers(0, 2 ** 14, sc.shape).astype(np.float32) * np.float32(2.0 ** -23))
    else:
        recent = W                                        # recent tokens fill the budget
    k, v, nsc, npos = _run_evict(pa, p, sc, pos, np.asarray(keep, np.int32), recent, False)
    assert pa.pa_device_status() == 0
    want = p.k.clone()
    for s, L in enumerate(lens):
        n = min(keep[s], L)
        src = _evict_ref(sc[s, 0, :L].astype(np.float64), pos[s, 0, :L], n, recent)
        assert np.array_equal(nsc[s, 0, :n], sc[s, 0, src], equal_nan=True), s
        assert np.array_equal(npos[s, 0, :n], pos[s, 0, src]), s
        i = np.arange(n)
        want[p.tables[s][i // 16], 0, i % 16] = p.k[p.tables[s][src // 16], 0, src % 16]
    assert np.array_equal(k.view(torch.int16).numpy(), want.view(torch.int16).numpy())


@pytest.mark.parametrize("Hkv,G,D", [(1, 8, 128), (2, 1, 64)])
def test_shared_extremes_of_groups(pa, Hkv, G, D):
    """Groups of one row, of none, of a thousand rows, and of every row of the batch."""
    p, q, groups = _batch(Hkv, G, D, 16, seed=60, groups=[(1, 20, [3]), (1000, 14, [0, 1, 2]), (2, 40, [500])], singles=[7])
    for listed in (groups[:1] + [([], 160)] + groups[1:], [([], 0)] + groups):
        out = shared_call(pa, p, q, listed, 0.1)
        assert pa.pa_device_status() == 0
        shared_check(p, q, out, 0.1, G)
    p, q, groups = _batch(Hkv, G, D, 16, seed=61, groups=[(70, 25, [0])], singles=[])
    out = shared_call(pa, p, q, groups, 0.1)
    assert pa.pa_device_status() == 0
    shared_check(p, q, out, 0.1, G)
