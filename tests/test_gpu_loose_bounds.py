"""pa_cross_attention with a max_query_len far above every sequence's rows: the same bits as with the rows' number."""
import numpy as np
import pytest
import torch

from pa_ops_testlib import Paged
from test_gpu_cross import _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hkv,G,D,lens,rows", [
    (8, 4, 128, [300, 500, 40, 700, 64, 90, 200, 10], [200, 130, 256, 90, 300, 257, 128, 300]),
    (2, 4, 128, [300, 500], [3, 1]), (2, 1, 64, [1000], [1]), (1, 8, 64, [90, 3000], [0, 40])])
def test_cross_bound_above_the_rows(Hkv, G, D, lens, rows):
    from paged_kv_cache_363_b200 import pa
    p = Paged(lens, Hkv, 16, D, torch.bfloat16, seed=len(lens))
    n = sum(rows)
    q = p.q(n, Hkv * G)
    k, v, tables, ctx = p.cuda()
    at = torch.from_numpy(np.cumsum([0] + rows).astype(np.int32)).cuda()
    got = []
    for most in (n, n + 1, 2 ** 20, 2 ** 31 - 1):
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        need = pa.pa_cross_attention_workspace_size(len(lens), Hkv * G, Hkv, D, 16, n, most, max(lens))
        assert need == pa.pa_cross_attention_workspace_size(len(lens), Hkv * G, Hkv, D, 16, n, n, max(lens))
        pa.pa_cross_attention(out, q.cuda(), k, v, tables, ctx, at, most, max(lens), D ** -0.5, lse=lse,
                              workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        assert pa.pa_device_status() == 0
        got.append((out, lse))
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    _check(p, rows, q, got[0][0], got[0][1], D ** -0.5, G)
