"""pa_evict on scores with NaN among finite ones, in every kind of storage that the selection has."""
import numpy as np
import pytest
import torch

from pa_ops_testlib import Paged
from pa_testlib import bits
from test_gpu_scores_evict import _evict_ref, _run_evict

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_363_b200 import pa as _pa
    return _pa


@pytest.mark.parametrize("Hkv,D,B,dt,lens", [
    (2, 64, 16, torch.bfloat16, [100, 1400, 257, 4096]),            # all cached, rows moved by a second kernel
    (75, 64, 16, torch.float32, [100, 1400]),                       # all cached, rows moved by the same kernel
    (1, 64, 32, torch.bfloat16, [5000, 100, 30000]),                # keys cached
    (1, 64, 32, torch.bfloat16, [50000, 1400])])                    # read again in every pass
@pytest.mark.parametrize("share,least", [(0.02, 0.1), (0.2, 1e-3), (0.93, 0.7), (0.2, 0.0), (0.2, -0.3), (0.93, 3.0)])
@pytest.mark.parametrize("recent", [0, 64])
def test_evict_nan_among_scores(pa, Hkv, D, B, dt, lens, share, least, recent):
    rng = np.random.default_rng(int(1000 * share) + recent)
    S, W = len(lens), max(lens)
    sc = np.maximum(np.exp(rng.standard_normal((S, Hkv, W))), abs(least)).astype(np.float32)
    pos = np.stack([np.stack([rng.permutation(W).astype(np.int32) for _ in range(Hkv)]) for _ in lens])
    for s, L in enumerate(lens):
        sc[s, :, int(rng.integers(L))] = least
        sc[s, :, :L][rng.random((Hkv, L)) < share] = np.nan
        for h in range(Hkv):
            pos[s, h, :L] = rng.permutation(L)
    p = Paged(lens, Hkv, B, D, dt, seed=7)
    # budgets on either side of the NaN tokens' number
    for at in (0.4, 0.98, 1.1, 3.0):
        keep = [max(1, min(L - 1, int(at * share * L) + (recent if at > 0.9 else 0))) for L in lens]
        k, v, nsc, npos = _run_evict(pa, p, sc, pos, np.asarray(keep, np.int32), recent, False)
        assert pa.pa_device_status() == 0
        want_k, want_v = p.k.clone(), p.v.clone()
        for s, L in enumerate(lens):
            n = keep[s]
            for h in range(Hkv):
                src = _evict_ref(sc[s, h, :L].astype(np.float64), pos[s, h, :L], n, recent)
                assert np.array_equal(nsc[s, h, :n], sc[s, h, src], equal_nan=True), (s, h)
                assert np.array_equal(npos[s, h, :n], pos[s, h, src]), (s, h)
                i = np.arange(n)
                d, f = (p.tables[s][i // B], i % B), (p.tables[s][src // B], src % B)
                want_k[d[0], h, d[1]], want_v[d[0], h, d[1]] = p.k[f[0], h, f[1]], p.v[f[0], h, f[1]]
        assert np.array_equal(bits(k), bits(want_k)) and np.array_equal(bits(v), bits(want_v))
