"""NaN in q, in a visible key or in a visible value: the rows and columns that see it become NaN on every path of
pa_cross_attention and pa_decode_shared, the others keep their bits."""
import numpy as np
import pytest
import torch

from pa_ops_testlib import Paged
from test_gpu_shared import _batch, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_363_b200 import pa as _pa
    return _pa


def _same(a, b):
    return a.view(torch.int16 if a.dtype == torch.bfloat16 else torch.int32).equal(
        b.view(torch.int16 if b.dtype == torch.bfloat16 else torch.int32))


def _poisoned(call, q, k, v, slot, seq_rows, row, G, D):
    """call(q, k, v) -> [out, lse or None].  slot: (block, offset) of a token of kv head 1 that the rows seq_rows see."""
    clean = call(q, k, v)
    heads = slice(G, 2 * G)
    # a query row, one head of it
    x = q.clone()
    x[row, G] = float("nan")
    got = call(x, k, v)
    assert bool(got[0][row, G].isnan().all())
    for i, (a, b) in enumerate(zip(got, clean)):
        if a is not None:
            assert bool(a[row, G].isnan().all())
            a[row, G] = b[row, G]
            assert _same(a, b)
    # a key
    x = k.clone()
    x[slot[0], 1, slot[1], D // 2] = float("nan")
    got = call(q, x, v)
    for a, b in zip(got, clean):
        if a is not None:
            assert bool(a[seq_rows, heads].isnan().all())
            a[seq_rows, heads] = b[seq_rows, heads]
            assert _same(a, b)
    # a value, whose column is D // 2 + 1
    x = v.clone()
    x[slot[0], 1, slot[1], D // 2 + 1] = float("nan")
    got = call(q, k, x)
    assert bool(got[0][seq_rows, heads, D // 2 + 1].isnan().all())
    got[0][seq_rows, heads, D // 2 + 1] = clean[0][seq_rows, heads, D // 2 + 1]
    assert _same(got[0], clean[0]) and (got[1] is None or _same(got[1], clean[1]))


@pytest.mark.parametrize("D,G", [(64, 1), (128, 4), (64, 8), (128, 2)])
@pytest.mark.parametrize("rows,top", [(1, 90), (1, 6000), (3, 90), (3, 6000), (0, 700)])
def test_cross_attention(pa, D, G, rows, top):
    """One row per sequence or three, whole contexts and split ones; 0: many rows, two query tiles at a time."""
    B, Hkv = 16, 8 if rows == 0 else 2
    rows = rows or 256 // G
    lens = [top // 3, top, 5, 17] + ([top] * 8 if rows > 3 else [])
    p = Paged(lens, Hkv, B, D, torch.bfloat16, seed=D + rows)
    n = len(lens) * rows
    q = p.q(n, Hkv * G).cuda()
    k, v, tables, ctx = p.cuda()
    at = _i32(np.arange(len(lens) + 1) * rows)

    def call(x, kk, vv):
        out, lse = torch.full_like(x, 7.0), torch.full((n, Hkv * G), 7.0, device="cuda")
        pa.pa_cross_attention(out, x, kk, vv, tables, ctx, at, rows, top, 0.2, lse=lse)
        torch.cuda.synchronize()
        assert pa.pa_device_status() == 0
        return [out, lse]

    for s in (1, 2):                             # the longest context, and one of five tokens
        for t in (lens[s] - 1, 0, lens[s] // 2):
            _poisoned(call, q, k, v, (int(p.tables[s][t // B]), t % B), slice(s * rows, (s + 1) * rows), s * rows + rows // 2, G, D)


@pytest.mark.parametrize("D,G", [(64, 1), (128, 4), (64, 8), (128, 2)])
@pytest.mark.parametrize("blocks,own", [(4, [1, 40]), (60, [1, 40, 0]), (300, [2500, 3])])
def test_decode_shared(pa, D, G, blocks, own):
    """Short contexts, which are read per row; groups; groups whose rows have long tokens of their own."""
    B, Hkv = 16, 2
    p, q, groups = _batch(Hkv, G, D, B, seed=80 + D, groups=[(6, blocks, own), (3, blocks // 2, [9])], singles=[100, 1, 0])
    rows, starts, lens = (_i32(sum([g for g, _ in groups], [])), _i32(np.cumsum([0] + [len(g) for g, _ in groups])),
                          _i32([n for _, n in groups]))
    k, v, tables, ctx = p.cuda()

    def call(x, kk, vv):
        out = torch.full_like(x, 7.0)
        pa.pa_decode_shared(out, x, kk, vv, tables, ctx, rows, starts, lens, max(p.lens), int(lens.max()), 0.2)
        torch.cuda.synchronize()
        assert pa.pa_device_status() == 0
        return [out, None]

    members = groups[0][0]
    s = members[0]
    for t in (0, 16 * blocks - 1):               # a shared token: every member sees it
        _poisoned(call, q.cuda(), k, v, (int(p.tables[s][t // B]), t % B), torch.tensor(members, device="cuda"), s, G, D)
    for s in [i for i in range(len(p.lens)) if p.lens[i] > 16 * blocks and i in members][:1] + [
            i for i in range(len(p.lens)) if p.lens[i] == 100][:1]:
        t = p.lens[s] - 1                        # a token of its own
        _poisoned(call, q.cuda(), k, v, (int(p.tables[s][t // B]), t % B), slice(s, s + 1), s, G, D)
