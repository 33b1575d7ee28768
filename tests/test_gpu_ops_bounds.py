"""The serving operators at the largest batches and contexts they take."""
import numpy as np
import pytest
import torch

from pa_ops_testlib import Paged, attend, output_tolerance
from test_gpu_scores_evict import _evict_ref, _run_evict

pytestmark = pytest.mark.gpu

MOST = 65535


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_363_b200 import pa as _pa
    return _pa


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def _pool(seed, NB=500, Hkv=1, B=16, D=64):
    rng = np.random.default_rng(seed)
    k, v = (torch.from_numpy(rng.standard_normal((NB, Hkv, B, D), dtype=np.float32)).to(torch.bfloat16) for _ in range(2))
    return rng, k, v


def _check_row(q, k, v, table, L, out, scale):
    i = np.arange(L)
    kk, vv = (x[table[i // 16], 0, i % 16].double().numpy().reshape(L, -1) for x in (k, v))
    o, pr, _, mags = attend(q.double().numpy(), kk, vv, scale)
    assert np.all(np.abs(out.float().cpu().double().numpy() - o) <= output_tolerance(pr, vv, o, mags, q.shape[-1]))


@pytest.mark.parametrize("most", [1, 2])
def test_cross_attention_of_the_most_sequences(pa, most):
    rng, k, v = _pool(most)
    tables = rng.integers(0, 500, (MOST, 4)).astype(np.int32)     # blocks may be anybody's: nothing is written
    ctx, rows = rng.integers(0, 65, MOST), rng.integers(0, most + 1, MOST)
    start = np.concatenate([[0], np.cumsum(rows)])
    q = torch.from_numpy(rng.standard_normal((int(start[-1]), 2, 64), dtype=np.float32)).to(torch.bfloat16)
    out, lse = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda"), torch.full(q.shape[:2], 7.0, device="cuda")
    pa.pa_cross_attention(out, q.cuda(), k.cuda(), v.cuda(), _i32(tables), _i32(ctx), _i32(start), most, 64, 0.125, lse=lse)
    torch.cuda.synchronize()
    assert pa.pa_device_status() == 0
    none = torch.from_numpy(np.repeat(ctx == 0, rows)).cuda()
    assert bool((out[none] == 0).all()) and bool((lse[none] == -np.inf).all()) and bool(lse[~none].isfinite().all())
    for s in [0, MOST - 1] + rng.integers(0, MOST, 300).tolist():
        for r in range(int(start[s]), int(start[s + 1])):
            if ctx[s]:
                _check_row(q[r], k, v, tables[s], int(ctx[s]), out[r], 0.125)


def test_decode_shared_of_the_most_sequences(pa):
    """32,767 pairs, most of which share a few blocks, long enough to be read per group."""
    rng, k, v = _pool(9)
    tables = rng.integers(0, 500, (MOST, 16)).astype(np.int32)
    order = rng.permutation(MOST).astype(np.int32)
    pairs = order[:2 * (MOST // 2)].reshape(-1, 2)
    shared = rng.integers(0, 12, len(pairs)) * 16
    for (a, b), n in zip(pairs, shared):
        tables[b, :n // 16] = tables[a, :n // 16]
    least = np.zeros(MOST, np.int64)
    least[pairs[:, 0]], least[pairs[:, 1]] = shared, shared
    ctx = np.minimum(256, least + rng.integers(0, 80, MOST))
    ctx[order[-1]] = 256
    q = torch.from_numpy(rng.standard_normal((MOST, 1, 64), dtype=np.float32)).to(torch.bfloat16)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    pa.pa_decode_shared(out, q.cuda(), k.cuda(), v.cuda(), _i32(tables), _i32(ctx), _i32(pairs.reshape(-1)),
                        _i32(np.arange(len(pairs) + 1) * 2), _i32(shared), 256, int(shared.max()), 0.125)
    plain = torch.empty_like(out)
    pa.pa_decode(plain, q.cuda(), k.cuda(), v.cuda(), _i32(tables), _i32(ctx), 256, 0.125)
    torch.cuda.synchronize()
    assert pa.pa_device_status() == 0
    # each side is within a weight's rounding of the definition
    most = float(v.float().abs().max())
    assert float((plain.float() - out.float()).abs().max()) <= most * 2.0 ** -8 + 2 * 2.0 ** -8 * float(plain.float().abs().max())
    for s in [int(order[-1]), 0, MOST - 1] + rng.integers(0, MOST, 300).tolist():
        if ctx[s]:
            _check_row(q[s], k, v, tables[s], int(ctx[s]), out[s], 0.125)


def test_scores_of_the_most_sequences(pa):
    rng, k, v = _pool(11)
    tables, ctx = rng.integers(0, 500, (MOST, 2)).astype(np.int32), rng.integers(0, 33, MOST)
    q = torch.from_numpy(rng.standard_normal((MOST, 2, 64), dtype=np.float32)).to(torch.bfloat16)
    out, sc = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda"), torch.zeros(MOST, 1, 32, device="cuda")
    pa.pa_decode_scores(out, sc, q.cuda(), k.cuda(), v.cuda(), _i32(tables), _i32(ctx), 32, 0.125)
    torch.cuda.synchronize()
    assert pa.pa_device_status() == 0
    # two heads' weights, each a sum of at most 32 terms that is divided by itself in fp32
    total = sc[:, 0].double().sum(-1).cpu().numpy()
    assert np.all(np.abs(total - 2 * (ctx > 0)) <= 2 * 64 * 2.0 ** -24)
    assert bool((sc[:, 0].cpu()[torch.arange(32)[None] >= torch.from_numpy(ctx)[:, None]] == 0).all())


@pytest.mark.parametrize("L,n", [(49152, 20000), (49153, 40000), (262144, 100001)])
def test_evict_of_the_longest_contexts(pa, L, n):
    p = Paged([L, 100], 1, 32, 64, torch.bfloat16, seed=L % 97)
    rng = np.random.default_rng(L)
    sc = np.exp(2 * rng.standard_normal((2, 1, L))).astype(np.float32)
    pos = np.stack([rng.permutation(L).astype(np.int32)[None] for _ in range(2)])
    pos[1, 0, :100] = rng.permutation(100)
    keep = np.asarray([n, 40], np.int32)
    k, v, nsc, npos = _run_evict(pa, p, sc, pos, keep, 333, False)
    assert pa.pa_device_status() == 0
    for s in range(2):
        src = _evict_ref(sc[s, 0, :p.lens[s]].astype(np.float64), pos[s, 0, :p.lens[s]], int(keep[s]), 333)
        assert np.array_equal(npos[s, 0, :keep[s]], pos[s, 0, src]) and np.array_equal(nsc[s, 0, :keep[s]], sc[s, 0, src])
        i = np.arange(int(keep[s]))
        for got, was in ((k, p.k), (v, p.v)):
            a = got[p.tables[s][i // 32], 0, i % 32].view(torch.int16)
            assert torch.equal(a, was[p.tables[s][src // 32], 0, src % 32].view(torch.int16))
