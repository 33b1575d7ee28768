"""Shapes that the bindings of the serving operators refuse before anything reaches the library (CPU only)."""
import pytest
import torch

pa = pytest.importorskip("paged_kv_cache_363_b200.pa", reason="libpa.so not built")

S, Hkv, G, D, B, NB, W = 3, 2, 2, 64, 16, 8, 40


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _cross(**over):
    a = dict(out=_bf16(5, Hkv * G, D), q=_bf16(5, Hkv * G, D), k_cache=_bf16(NB, Hkv, B, D), v_cache=_bf16(NB, Hkv, B, D),
             block_tables=_i32(S, 4), context_lens=_i32(S), q_start=_i32(S + 1), max_query_len=3, max_context_len=W, scale=1.0)
    pa.pa_cross_attention(**{**a, **over})


def _evict(**over):
    a = dict(k_cache=_bf16(NB, Hkv, B, D), v_cache=_bf16(NB, Hkv, B, D), new_scores=torch.zeros(S, Hkv, W),
             new_positions=_i32(S, Hkv, W), scores=torch.zeros(S, Hkv, W), positions=_i32(S, Hkv, W), block_tables=_i32(S, 4),
             context_lens=_i32(S), keep_lens=_i32(S), num_recent=2, max_context_len=W)
    pa.pa_evict(**{**a, **over})


@pytest.mark.parametrize("call,over", [
    (_cross, dict(context_lens=_i32(S, 2))), (_cross, dict(context_lens=_i32(S + 1))), (_cross, dict(q_start=_i32(S))),
    (_cross, dict(block_tables=_i32(S - 1, 4))), (_cross, dict(out=_bf16(4, Hkv * G, D))),
    (_cross, dict(v_cache=_bf16(NB, Hkv, B, 128))), (_cross, dict(lse=torch.zeros(5, Hkv))),
    (_evict, dict(context_lens=_i32(S, 2))), (_evict, dict(keep_lens=_i32(S, 1))), (_evict, dict(block_tables=_i32(S * 4))),
    (_evict, dict(positions=_i32(S, Hkv, W + 1))), (_evict, dict(v_cache=_bf16(NB, Hkv, B, 128)))])
def test_shapes(call, over):
    with pytest.raises(ValueError):
        call(**over)


@pytest.mark.parametrize("call,over", [
    (_cross, dict(context_lens=torch.zeros(S, dtype=torch.int64))), (_cross, dict(q=torch.zeros(5, Hkv * G, D))),
    (_evict, dict(keep_lens=torch.zeros(S, dtype=torch.int64))), (_evict, dict(scores=torch.zeros(S, Hkv, W, dtype=torch.float64))),
    (_evict, dict(v_cache=torch.zeros(NB, Hkv, B, D)))])
def test_types(call, over):
    with pytest.raises(TypeError):
        call(**over)
