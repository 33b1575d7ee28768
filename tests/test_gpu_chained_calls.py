"""pa_decode_run behind calls whose output is its q, with no other kernel between them: the same bits as with a wait
between the calls."""
import numpy as np
import pytest
import torch

from pa_ops_testlib import Paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_363_b200 import pa as _pa
    return _pa


@pytest.mark.parametrize("kind", ["run", "decode", "scores", "cross", "shared"])
@pytest.mark.parametrize("G,D,S,top", [(4, 128, 30, 500), (1, 128, 60, 300), (8, 64, 9, 4000)])
def test_run_takes_the_last_call_s_output(pa, kind, G, D, S, top):
    Hkv, B = 4, 16
    rng = np.random.default_rng(S)
    lens = rng.integers(1, top + 1, S).tolist()
    p = Paged(lens, Hkv, B, D, torch.bfloat16, seed=S)
    k, v, tables, ctx = p.cuda()
    q = p.q(S, Hkv * G).cuda()
    mx = max(lens)
    sizes = (S, Hkv * G, Hkv, D, B)
    ws = torch.empty(pa.pa_decode_workspace_size(*sizes, mx), dtype=torch.uint8, device="cuda")
    need = max(pa.pa_decode_workspace_size(*sizes, mx), pa.pa_decode_scores_workspace_size(*sizes, mx),
               pa.pa_cross_attention_workspace_size(*sizes, S, 2, mx), pa.pa_decode_shared_workspace_size(*sizes, mx, 0, 0, 0))
    ws2 = torch.empty(need, dtype=torch.uint8, device="cuda")
    start = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_decode_plan(tables, ctx, mx, Hkv * G, k, ws)

    def before(out, x, scores):
        if kind == "run":
            pa.pa_decode_run(out, x, k, v, tables, ctx, mx, 0.5, ws)
        elif kind == "decode":
            pa.pa_decode(out, x, k, v, tables, ctx, mx, 0.5, workspace=ws2)
        elif kind == "scores":
            pa.pa_decode_scores(out, scores, x, k, v, tables, ctx, mx, 0.5, workspace=ws2)
        elif kind == "cross":
            pa.pa_cross_attention(out, x, k, v, tables, ctx, start, 2, mx, 0.5, workspace=ws2)
        else:
            pa.pa_decode_shared(out, x, k, v, tables, ctx, none[:0], none, none[:0], mx, 0, 0.5, workspace=ws2)

    def chain(wait):
        # two buffers: a call's output takes the place of the q before the last one
        a, b = q.clone(), torch.zeros_like(q)
        scores = torch.zeros(S, Hkv, mx, device="cuda")
        torch.cuda.synchronize()
        for _ in range(12):
            before(b, a, scores)
            if wait:
                torch.cuda.synchronize()
            pa.pa_decode_run(a, b, k, v, tables, ctx, mx, 0.5, ws)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return a, b, scores

    want = chain(True)
    for _ in range(5):
        got = chain(False)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert pa.pa_device_status() == 0
