"""Block tables whose rows have room for 2^31 tokens and more: the same bits as with a narrow table."""
import numpy as np
import pytest
import torch

from pa_ops_testlib import Paged

pytestmark = pytest.mark.gpu


def test_rows_with_room_for_two_to_the_31_tokens():
    from paged_kv_cache_363_b200 import pa
    Hkv, G, D, B, L = 2, 4, 128, 16, 1000
    p = Paged([L], Hkv, B, D, torch.bfloat16, seed=1)
    k, v, tables, ctx = p.cuda()
    wide = torch.full((1, 2 ** 27 + 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :tables.shape[1]] = tables
    q, few = p.q(1, Hkv * G).cuda(), p.q(3, Hkv * G).cuda()
    many = p.q(6400, Hkv * G).cuda()            # enough tiles of rows to share them
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    sc = torch.rand(1, Hkv, L, device="cuda")
    pos = torch.arange(L, dtype=torch.int32, device="cuda").expand(1, Hkv, L).contiguous()

    def run(t):
        o = [torch.full_like(x, 7.0) for x in (q, q, q, few, many, few, q)]
        pa.pa_decode(o[0], q, k, v, t, ctx, L, 0.1)
        s = sc.clone()
        pa.pa_decode_scores(o[1], s, q, k, v, t, ctx, L, 0.1)
        pa.pa_decode_shared(o[2], q, k, v, t, ctx, i32([0]), i32([0, 1]), i32([800]), L, 800, 0.1)
        pa.pa_cross_attention(o[6], q, k, v, t, ctx, i32([0, 1]), 1, L, 0.1)
        pa.pa_cross_attention(o[3], few, k, v, t, ctx, i32([0, 3]), 3, L, 0.1)
        pa.pa_cross_attention(o[4], many, k, v, t, ctx, i32([0, 6400]), 6400, L, 0.1)
        pa.pa_prefill(o[5], few, k, v, t, ctx, i32([0, 3]), 3, 0.1)
        kk, vv, ns, npos = k.clone(), v.clone(), torch.zeros_like(sc), torch.zeros_like(pos)
        pa.pa_evict(kk, vv, ns, npos, sc, pos, t, ctx, i32([300]), 16, L)
        torch.cuda.synchronize()
        assert pa.pa_device_status() == 0
        return o + [s, kk.nan_to_num(9.0), vv.nan_to_num(9.0), ns, npos]

    for a, b in zip(run(tables), run(wide)):
        assert torch.equal(a, b)
    assert int(np.count_nonzero(wide[0, tables.shape[1]:tables.shape[1] + 9].cpu() + 1)) == 0
