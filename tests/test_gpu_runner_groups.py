"""The batches' decode_shared when the allocator has moved on since the last call."""
import numpy as np
import pytest
import torch

from paged_kv_cache_363_b200 import runner, workloads as W

pytestmark = pytest.mark.gpu


def _rebuild(b):
    S = b.wl.num_seqs
    mb = max(len(b.alloc.block_table(s)) for s in range(S))
    tables, ctx = b.alloc.block_tables(np.arange(S), mb, fill=-1)
    b.block_tables, b.context_lens = torch.from_numpy(tables).to(b.device), torch.from_numpy(ctx).to(b.device)
    b.max_context_len = int(ctx.max())
    b.workspace_for(b.partition_size)


def _compare(pa, b, stream=None, groups=None):
    plain = b.decode(out=torch.empty_like(b.out)).float()
    out = torch.full_like(b.out, 7.0)
    torch.cuda.synchronize()
    b.decode_shared(out=out, stream=stream, **({} if groups is None else {"groups": groups}))
    torch.cuda.synchronize()
    assert pa.pa_device_status() == 0
    # each side is within a weight's rounding of the definition; values of V are below 6
    assert float((plain - out.float()).abs().max()) <= 6 * 2.0 ** -8 + 2 * 2.0 ** -8 * float(plain.abs().max())


def _batch():
    wl = W.make_workload(4, seed=2, num_prompts=4, streams_per_prompt=3, prompt_lens=(200, 400), private_tokens=(1, 30),
                         num_blocks=900)
    b = runner.make_batch(wl, "cuda")
    b.append()
    return b


def test_groups_follow_private_copies_and_shorter_sequences():
    from paged_kv_cache_363_b200 import pa
    b = _batch()
    _compare(pa, b)
    B = b.wl.block_size
    # one stream of each prompt takes its first blocks for itself and changes them
    for s in range(0, b.wl.num_seqs, 3):
        pairs = b.alloc.make_private(s, 5 * B)
        assert len(pairs) == 5
        own = torch.from_numpy(pairs[:, 1].copy()).to(b.device)
        b.v_cache[own] = torch.randn(5, *b.v_cache.shape[1:], device=b.device).clamp(-5, 5).to(b.v_cache.dtype)
        b.k_cache[own] = torch.randn(5, *b.k_cache.shape[1:], device=b.device).to(b.k_cache.dtype)
    _rebuild(b)
    _compare(pa, b)
    for s in range(1, b.wl.num_seqs, 3):
        b.alloc.truncate(s, 3 * B)
    _rebuild(b)
    _compare(pa, b, stream=torch.cuda.Stream())


def test_workspace_grows_with_the_batch_and_a_step_is_captured():
    from paged_kv_cache_363_b200 import pa
    b = _batch()
    for s in range(b.wl.num_seqs):
        b.alloc.truncate(s, 32)
    _rebuild(b)
    _compare(pa, b)
    small = b.shared_workspace.numel()
    b = _batch()
    b.shared_workspace = torch.empty(small, dtype=torch.uint8, device=b.device)
    _compare(pa, b)
    assert b.shared_workspace.numel() > small
    groups = b.shared_groups()
    _compare(pa, b, groups=groups)
    out = torch.empty_like(b.out)
    want = b.decode_shared(groups=groups).clone()
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        b.decode_shared(out=out, stream=side, groups=groups)
    out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_a_step_captured_after_a_call():
    """Without `groups`: those of the call before, which the graph keeps; refused where they are not the batch's any more."""
    from paged_kv_cache_363_b200 import pa
    b = _batch()
    want = b.decode_shared().clone()
    torch.cuda.synchronize()
    out = torch.empty_like(b.out)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        b.decode_shared(out=out, stream=side)
    b.shared_workspace = None
    for _ in range(3):                       # other calls, whose groups and workspace are their own
        b.decode_shared(out=torch.empty_like(b.out))
    junk = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in (64, 512, 512, 4096, 1 << 20)]
    out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    assert pa.pa_device_status() == 0
    assert torch.equal(out, want) and len(junk) == 5
    b = _batch()
    with pytest.raises(ValueError):
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):
            b.decode_shared(out=out, stream=side)
    torch.cuda.synchronize()
    _compare(pa, b)
