"""pa_cross_attention on the GPU against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from pa_ops_testlib import EPS32, Paged, attend, logit_error, output_tolerance
from pa_testlib import bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_363_b200 import pa as _pa
    return _pa


def _check(p, rows, q, out, lse, scale, G):
    start = np.concatenate([[0], np.cumsum(rows)])
    out, lse = out.float().cpu().double().numpy(), lse.cpu().double().numpy()
    for s, L in enumerate(p.lens):
        a, b = start[s], start[s + 1]
        if a == b:
            continue
        for h in range(p.Hkv):
            k, v = p.rows(s, h)
            qq = q[a:b, h * G:(h + 1) * G].double().numpy().reshape(-1, p.D)
            o, pr, z, mags = attend(qq, k, v, scale)
            got = out[a:b, h * G:(h + 1) * G].reshape(-1, p.D)
            zl = lse[a:b, h * G:(h + 1) * G].reshape(-1)
            if L == 0:
                assert np.all(got == 0) and np.all(zl == -np.inf)
                continue
            assert np.all(np.abs(got - o) <= output_tolerance(pr, v, o, mags, p.D)), (s, h, np.abs(got - o).max())
            assert np.all(np.abs(zl - z) <= 2 * logit_error(mags, p.D).max() + 64 * EPS32 * (1 + np.abs(z))), (s, h)


def _call(pa, p, rows, q, scale, ws=None, stream=None):
    k, v, tables, ctx = p.cuda()
    start = torch.from_numpy(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)).cuda()
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    pa.pa_cross_attention(out, q.cuda(), k, v, tables, ctx, start, max(rows), max(max(p.lens), 1), scale, lse=lse,
                          workspace=ws, stream=stream)
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("Hkv,G,D,B", [(2, 1, 128, 16), (1, 2, 64, 32), (2, 4, 128, 32), (1, 8, 128, 16),
                                       (3, 1, 64, 16), (2, 4, 64, 16), (1, 8, 64, 32), (1, 2, 128, 16)])
def test_cross_against_the_definition(pa, Hkv, G, D, B):
    lens = [1, 0, 15, 16, 17, 63, 64, 65, 128, 129, 700, 33, 5]
    rows = [1, 3, 2, 0, 31, 32, 33, 1, 130, 1, 65, 0, 17]
    p = Paged(lens, Hkv, B, D, torch.bfloat16, seed=Hkv * 100 + G * D + B)
    q = p.q(sum(rows), Hkv * G)
    out, lse = _call(pa, p, rows, q, D ** -0.5)
    assert pa.pa_device_status() == 0
    _check(p, rows, q, out, lse, D ** -0.5, G)


@pytest.mark.parametrize("Hkv,G,D,B", [(2, 1, 128, 16), (1, 2, 64, 32), (2, 4, 128, 32), (1, 8, 128, 16), (3, 1, 64, 16),
                                       (2, 4, 64, 16), (1, 8, 64, 32)])
def test_cross_single_rows(pa, Hkv, G, D, B):
    """At most one query row per sequence, some without one and some without tokens, long ones in parts."""
    lens = [1, 0, 15, 16, 17, 0, 64, 65, 300, 1029, 5000, 33, 5]
    rows = [1, 1, 0, 1, 1, 0, 1, 1, 1, 1, 1, 0, 1]
    p = Paged(lens, Hkv, B, D, torch.bfloat16, seed=Hkv + G * D + B)
    q = p.q(sum(rows), Hkv * G)
    for scale in (D ** -0.5, -0.3):
        out, lse = _call(pa, p, rows, q, scale)
        assert pa.pa_device_status() == 0
        _check(p, rows, q, out, lse, scale, G)


def test_cross_single_rows_many_and_bad(pa):
    rng = np.random.default_rng(3)
    S = 1500                                              # more sequences than plan threads
    lens, rows = rng.integers(0, 300, S).tolist(), rng.integers(0, 2, S).tolist()
    p = Paged(lens, 1, 16, 64, torch.bfloat16, seed=23)
    q = p.q(sum(rows), 2)
    out, lse = _call(pa, p, rows, q, 0.125)
    assert pa.pa_device_status() == 0
    _check(p, rows, q, out, lse, 0.125, 2)
    k, v, tables, ctx = p.cuda()
    start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    s = int(np.flatnonzero(np.array(rows) == 1)[7])
    ctx[s] = 10 ** 6                                      # a context past its table
    out2 = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    pa.pa_cross_attention(out2, q.cuda(), k, v, tables, ctx, torch.from_numpy(start).cuda(), 1, max(lens), 0.125)
    torch.cuda.synchronize()
    assert pa.pa_device_status() == pa.PA_DEV_BAD_CONTEXT
    good = [i for i in range(len(q)) if i != start[s]]
    assert torch.equal(out2[good], out[good]) and torch.all(out2[start[s]] == 7.0)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 2.0])
def test_cross_scales(pa, scale):
    """A negative scale, none, and one that makes the softmax sharp (running maxima that grow far)."""
    lens, rows = [300, 65, 1000], [20, 3, 1]
    p = Paged(lens, 2, 16, 128, torch.bfloat16, seed=8)
    q = p.q(sum(rows), 4)
    # keys that grow along the sequence, so that later tiles raise the maximum by more than 8
    ramp = torch.linspace(0.1, 3.0, p.width)
    for s in range(3):
        for i in range(-(-lens[s] // 16)):
            p.k[p.tables[s, i]] *= ramp[i]
    out, lse = _call(pa, p, rows, q, scale)
    assert pa.pa_device_status() == 0
    _check(p, rows, q, out, lse, scale, 2)


def test_cross_long_tables_in_chunks(pa):
    """One query row against 20,000 tokens, beside short ones: the tokens are split and joined."""
    lens, rows = [20011, 300, 9000], [1, 40, 2]
    p = Paged(lens, 1, 32, 64, torch.bfloat16, seed=10)
    q = p.q(sum(rows), 4)
    out, lse = _call(pa, p, rows, q, 0.125)
    assert pa.pa_device_status() == 0
    _check(p, rows, q, out, lse, 0.125, 4)


def test_cross_many_short_sequences(pa):
    """More units than the grid holds at once, each of one or two tiles."""
    rng = np.random.default_rng(1)
    S = 700
    lens, rows = rng.integers(0, 130, S).tolist(), rng.integers(0, 9, S).tolist()
    p = Paged(lens, 2, 16, 64, torch.bfloat16, seed=12)
    q = p.q(sum(rows), 4)
    out, lse = _call(pa, p, rows, q, 0.125)
    assert pa.pa_device_status() == 0
    _check(p, rows, q, out, lse, 0.125, 2)


@pytest.mark.parametrize("Hkv,G,D", [(2, 4, 128), (4, 1, 64), (1, 8, 128)])
def test_cross_many_rows(pa, Hkv, G, D):
    lens, rows = [900, 257, 1, 640], [700, 129, 300, 513]
    p = Paged(lens, Hkv, 16, D, torch.bfloat16, seed=D + G)
    q = p.q(sum(rows), Hkv * G)
    out, lse = _call(pa, p, rows, q, D ** -0.5)
    assert pa.pa_device_status() == 0
    _check(p, rows, q, out, lse, D ** -0.5, G)


# Enough rows that two tiles of 128 query rows share every K/V tile (head_dim 128).
SHARED_TILES = [(2, 8, 16, [700, 0, 1, 129, 64, 257], [300, 70, 130, 0, 200, 150]),
                (8, 1, 32, [1, 300, 63, 0, 31], [515, 257, 384, 260, 400]),
                (4, 4, 16, [2000, 5, 0, 128], [129, 400, 33, 300]),
                (8, 2, 16, [65, 17, 0, 511], [300, 200, 1, 399])]


@pytest.mark.parametrize("Hkv,G,B,lens,rows", SHARED_TILES)
@pytest.mark.parametrize("scale", [128 ** -0.5, -0.1, 0.0])
def test_cross_rows_that_share_tiles(pa, Hkv, G, B, lens, rows, scale):
    p = Paged(lens, Hkv, B, 128, torch.bfloat16, seed=31 + G)
    q = p.q(sum(rows), Hkv * G)
    out, lse = _call(pa, p, rows, q, scale)
    assert pa.pa_device_status() == 0
    _check(p, rows, q, out, lse, scale, G)


def test_cross_rows_that_share_tiles_skip_bad_sequences_and_replay(pa):
    Hkv, G, B, lens, rows = SHARED_TILES[2]
    p = Paged(lens, Hkv, B, 128, torch.bfloat16, seed=33)
    q = p.q(sum(rows), Hkv * G)
    good, _ = _call(pa, p, rows, q, 0.1)
    k, v, tables, ctx = p.cuda()
    qd, start = q.cuda(), torch.from_numpy(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)).cuda()
    nbytes = pa.pa_cross_attention_workspace_size(4, Hkv * G, Hkv, 128, B, sum(rows), max(rows), 2000)
    ws = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
    side, outs, graphs = torch.cuda.Stream(), [torch.empty_like(qd) for _ in range(2)], []
    side.wait_stream(torch.cuda.current_stream())
    for o in outs:                                        # two graphs that share a workspace, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            pa.pa_cross_attention(o, qd, k, v, tables, ctx, start, max(rows), 2000, 0.1, workspace=ws, stream=side)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert pa.pa_device_status() == 0
    assert all(torch.equal(o, good) for o in outs)
    a = np.concatenate([[0], np.cumsum(rows)])
    for s, L in ((0, 10 ** 6), (1, -3), (3, 129 + 10 ** 5)):
        c = ctx.clone()
        c[s] = L
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        pa.pa_cross_attention(out, qd, k, v, tables, c, start, max(rows), 2000, 0.1)
        torch.cuda.synchronize()
        assert pa.pa_device_status() == pa.PA_DEV_BAD_CONTEXT
        assert torch.all(out[a[s]:a[s + 1]] == 7.0)
        rest = [i for i in range(len(q)) if not a[s] <= i < a[s + 1]]
        assert torch.equal(out[rest], good[rest])


def test_cross_captured_on_another_stream_and_shared_workspace(pa):
    lens, rows = [333, 64, 2000], [3, 200, 1]
    p = Paged(lens, 2, 16, 128, torch.bfloat16, seed=14)
    q = p.q(sum(rows), 8)
    first, lse0 = _call(pa, p, rows, q, 0.1)
    k, v, tables, ctx = p.cuda()
    qd = q.cuda()
    start = torch.from_numpy(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)).cuda()
    ws = torch.full((pa.pa_cross_attention_workspace_size(3, 8, 2, 128, 16, sum(rows), 200, 2000),), 255,
                    dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(qd) for _ in range(2)]
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for o in outs:                                        # two graphs that share a workspace, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            pa.pa_cross_attention(o, qd, k, v, tables, ctx, start, 200, 2000, 0.1, workspace=ws, stream=side)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert pa.pa_device_status() == 0
    for o in outs:
        assert np.array_equal(bits(o), bits(first))       # chunking and order do not depend on the run


def test_cross_flags_and_skips_bad_sequences(pa):
    lens, rows = [100, 90, 80, 70], [5, 6, 7, 8]
    p = Paged(lens, 1, 16, 64, torch.bfloat16, seed=15)
    q = p.q(sum(rows), 2)
    good, _ = _call(pa, p, rows, q, 0.125)
    k, v, tables, ctx = p.cuda()
    for start, ctxs, skipped in (([0, 5, 11, 18, 40], lens, [3]), ([0, 5, 3, 18, 26], lens, [1, 2]),
                                 ([-1, 5, 11, 18, 26], lens, [0]), ([0, 5, 11, 18, 26], [100, -1, 10 ** 6, 70], [1, 2]),
                                 ([0, 5, 11, 18, 26], [100, 90, 113, 70], [2])):
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        # rows [11, 18) belong to sequence 2 unless the starts say otherwise
        pa.pa_cross_attention(out, q.cuda(), k, v, tables, torch.tensor(ctxs, dtype=torch.int32).cuda(),
                              torch.tensor(start, dtype=torch.int32).cuda(), 8, 112, 0.125)
        torch.cuda.synchronize()
        assert pa.pa_device_status() == pa.PA_DEV_BAD_CONTEXT
        for s in range(4):
            a, b = sum(rows[:s]), sum(rows[:s + 1])
            if s in skipped and start != [0, 5, 3, 18, 26]:
                assert torch.all(out[a:b] == 7.0)
            elif s not in skipped:
                assert torch.equal(out[a:b], good[a:b])
    p.tables[1, 2] = 10 ** 6                              # a block outside the pool: flagged
    k, v, tables, ctx = p.cuda()
    st = torch.tensor([0, 5, 11, 18, 26], dtype=torch.int32).cuda()
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    pa.pa_cross_attention(out, q.cuda(), k, v, tables, ctx, st, 8, 112, 0.125)
    torch.cuda.synchronize()
    assert pa.pa_device_status() == pa.PA_DEV_BAD_BLOCK
    assert torch.equal(out[:5], good[:5]) and torch.equal(out[11:], good[11:])


@pytest.mark.parametrize("Hkv,G,D,lens,rows", [
    (2, 4, 128, [200] * 100, [100] * 100), (1, 4, 128, [8192] * 4, [100] * 4), (4, 1, 64, [900, 257, 1, 640], [700, 129, 300, 513]),
    (8, 4, 128, [1, 900] * 20, [100] * 40)])
def test_cross_same_bits_in_every_run(pa, Hkv, G, D, lens, rows):
    """All four softmax warps busy, two CTAs per SM, warps that run ahead of each other: nothing may depend on it."""
    p = Paged(lens, Hkv, 16, D, torch.bfloat16, seed=21)
    q = p.q(sum(rows), Hkv * G).cuda()
    k, v, tables, ctx = p.cuda()
    start = torch.from_numpy(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)).cuda()
    outs = []
    for _ in range(25):
        out = torch.empty_like(q)
        pa.pa_cross_attention(out, q, k, v, tables, ctx, start, max(rows), max(lens), D ** -0.5)
        outs.append(out)
    torch.cuda.synchronize()
    assert pa.pa_device_status() == 0
    assert all(torch.equal(o, outs[0]) for o in outs)
