"""The serving operators called by two host threads at once, each on a stream and a workspace of its own."""
import threading

import numpy as np
import pytest
import torch

from pa_ops_testlib import Paged
from test_gpu_scores_evict import _evict_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_363_b200 import pa as _pa
    return _pa


@pytest.mark.parametrize("lens", [(5000, 45000), (300, 4096), (50000, 60000)])
def test_evict_from_two_threads(pa, lens):
    """Contexts whose kernels are the same and need different amounts of shared memory."""
    S, D, B, calls = 2, 64, 16, 400
    jobs = []
    for i, L in enumerate(lens):
        p = Paged([L] * S, 1, B, D, torch.bfloat16, seed=i)
        k, v, tables, ctx = p.cuda()
        rng = np.random.default_rng(i)
        sc = np.exp(rng.standard_normal((S, 1, L))).astype(np.float32)
        pos = np.tile(np.arange(L, dtype=np.int32), (S, 1, 1))
        n = L // 3
        a, b = torch.from_numpy(sc).cuda(), torch.from_numpy(pos).cuda()
        jobs.append(dict(k=k, v=v, tables=tables, ctx=ctx, sc=a, pos=b, nsc=torch.empty_like(a), npos=torch.empty_like(b), L=L,
                         keep=torch.full((S,), n, dtype=torch.int32, device="cuda"), stream=torch.cuda.Stream(),
                         ws=torch.empty(pa.pa_evict_workspace_size(S, 1, L), dtype=torch.uint8, device="cuda"),
                         want=[pos[s, 0, _evict_ref(sc[s, 0].astype(np.float64), pos[s, 0], n, 8)] for s in range(S)]))
    torch.cuda.synchronize()
    start, failures = threading.Barrier(2), []

    def work(j):
        try:
            start.wait()
            for _ in range(calls):
                pa.pa_evict(j["k"], j["v"], j["nsc"], j["npos"], j["sc"], j["pos"], j["tables"], j["ctx"], j["keep"], 8, j["L"],
                            workspace=j["ws"], stream=j["stream"])
        except Exception as e:  # noqa: BLE001
            failures.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failures
    assert pa.pa_device_status() == 0
    for j in jobs:
        for s in range(S):
            assert np.array_equal(j["npos"][s, 0, :len(j["want"][s])].cpu().numpy(), j["want"][s])
