"""Batches without a single token, whose scores and tables are empty arrays: zero rows, as with room that nothing uses."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,G,D", [("bf16", 4, 128), ("f32", 1, 64)])
def test_scores_of_no_tokens(dt, G, D):
    from paged_kv_cache_363_b200 import pa
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    S, Hkv = 3, 2
    k = torch.full((4, Hkv, 16, D), float("nan"), dtype=t, device="cuda")
    q = torch.randn(S, Hkv * G, D, device="cuda").to(t)
    out = torch.full_like(q, 7.0)
    ctx = torch.zeros(S, dtype=torch.int32, device="cuda")
    tables = torch.full((S, 1), -1, dtype=torch.int32, device="cuda")
    pa.pa_decode_scores(out, torch.empty(S, Hkv, 0, device="cuda"), q, k, k.clone(), tables, ctx, 0, 0.1)
    torch.cuda.synchronize()
    assert pa.pa_device_status() == 0
    assert bool((out == 0).all())


@pytest.mark.parametrize("rows,Hkv,G,D", [(1, 2, 4, 128), (3, 2, 1, 64), (64, 16, 4, 128)])
def test_cross_attention_to_no_tokens(rows, Hkv, G, D):
    from paged_kv_cache_363_b200 import pa
    S = 8
    k = torch.full((4, Hkv, 16, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = torch.randn(S * rows, Hkv * G, D, device="cuda").to(torch.bfloat16)
    out, lse = torch.full_like(q, 7.0), torch.full((S * rows, Hkv * G), 7.0, device="cuda")
    ctx = torch.zeros(S, dtype=torch.int32, device="cuda")
    start = torch.arange(S + 1, dtype=torch.int32, device="cuda") * rows
    pa.pa_cross_attention(out, q, k, k.clone(), torch.empty(S, 0, dtype=torch.int32, device="cuda"), ctx, start, rows, 0, 0.1,
                          lse=lse)
    torch.cuda.synchronize()
    assert pa.pa_device_status() == 0
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all())
