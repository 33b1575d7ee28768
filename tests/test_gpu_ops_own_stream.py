"""Calls on a stream that is not the current one, without a workspace: what the call allocates for itself belongs to that
stream."""
import numpy as np
import pytest
import torch

from test_gpu_shared import _batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_363_b200 import pa as _pa
    return _pa


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def _calls(pa):
    """name -> f(stream), which gives the call's outputs."""
    Hkv, G, D, B = 2, 4, 128, 16
    p, q, groups = _batch(Hkv, G, D, B, seed=70, groups=[(6, 40, [1, 40]), (3, 3, [200])], singles=[1000, 700, 1])
    rows, starts, lens = (_i32(sum([g for g, _ in groups], [])), _i32(np.cumsum([0] + [len(g) for g, _ in groups])),
                          _i32([n for _, n in groups]))
    k, v, tables, ctx = p.cuda()
    q = q.cuda()
    S, mx, most = q.shape[0], max(p.lens), int(lens.max())
    few = q.repeat_interleave(3, 0)
    scores = torch.rand(S, Hkv, mx, device="cuda")
    pos = torch.arange(mx, dtype=torch.int32, device="cuda").expand(S, Hkv, mx).contiguous()
    # eviction of sequences of its own: blocks 40 * i ...
    ek = torch.randn(4 * 40, Hkv, B, D, device="cuda").to(torch.bfloat16)
    et, ec, en = _i32(np.arange(160).reshape(4, 40)), _i32([640, 333, 17, 500]), _i32([100, 90, 16, 400])
    es = torch.rand(4, Hkv, 640, device="cuda")
    ep = pos[:4, :, :640].contiguous()
    start = _i32(np.arange(S + 1))

    def decode(stream):
        o = torch.full_like(q, 7.0)
        return [o], lambda: pa.pa_decode(o, q, k, v, tables, ctx, mx, 0.1, stream=stream)

    def shared(stream):
        o = torch.full_like(q, 7.0)
        return [o], lambda: pa.pa_decode_shared(o, q, k, v, tables, ctx, rows, starts, lens, mx, most, 0.1, stream=stream)

    def cross(x, n):
        at = start * n

        def f(stream):
            o = torch.full_like(x, 7.0)
            return [o], lambda: pa.pa_cross_attention(o, x, k, v, tables, ctx, at, n, mx, 0.1, stream=stream)
        return f

    def with_scores(stream):
        o, sc = torch.full_like(q, 7.0), scores.clone()
        return [o, sc], lambda: pa.pa_decode_scores(o, sc, q, k, v, tables, ctx, mx, 0.1, stream=stream)

    def evict(stream):
        a, b, ns, np_ = ek.clone(), ek.clone(), torch.zeros_like(es), torch.zeros_like(ep)
        return [a, b, ns, np_], lambda: pa.pa_evict(a, b, ns, np_, es, ep, et, ec, en, 8, 640, stream=stream)

    return {"decode": decode, "shared": shared, "cross one": cross(q, 1), "cross few": cross(few, 3), "scores": with_scores,
            "evict": evict}


@pytest.mark.parametrize("name", ["decode", "shared", "cross one", "cross few", "scores", "evict"])
def test_workspace_of_a_call_on_another_stream(pa, name, monkeypatch):
    f = _calls(pa)[name]
    want, call = f(None)
    call()
    torch.cuda.synchronize()
    made = []
    empty = torch.empty

    def spy(*args, **kw):
        t = empty(*args, **kw)
        if kw.get("dtype") == torch.uint8:
            made.append((t.data_ptr(), t.numel()))
        return t

    other = torch.cuda.Stream()
    for _ in range(3):
        got, call = f(other)
        torch.cuda.synchronize()
        # memory that the current stream has just let go of, and still writes to
        idle = [empty(1 << 20, dtype=torch.uint8, device="cuda") for _ in range(8)]
        torch.cuda._sleep(2_000_000)
        for t in idle:
            t.zero_()
        busy = [t.data_ptr() for t in idle]
        del idle, t
        with torch.cuda.stream(other):
            torch.cuda._sleep(2_000_000)
        monkeypatch.setattr(torch, "empty", spy)
        call()
        monkeypatch.setattr(torch, "empty", empty)
        ptr, n = made.pop()
        assert not made
        assert all(b + (1 << 20) <= ptr or ptr + n <= b for b in busy)
        # what the current stream allocates next, while the call runs, is other memory
        after = [empty(n, dtype=torch.uint8, device="cuda") for _ in range(4)]
        assert all(t.data_ptr() + n <= ptr or ptr + n <= t.data_ptr() for t in after)
        for t in after:
            t.zero_()
        torch.cuda.synchronize()
        assert pa.pa_device_status() == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del after, t
