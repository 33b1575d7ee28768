"""pa_decode_shared on the GPU against the definition in 64 bits, and through the batches whose
sequences share blocks (prefix cache, parallel sampling, beam search)."""
import numpy as np
import pytest
import torch

from pa_ops_testlib import Paged, attend, output_tolerance
from pa_testlib import bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_363_b200 import pa as _pa
    return _pa


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def _check(p, q, out, scale, G):
    out = out.float().cpu().double().numpy()
    for s, L in enumerate(p.lens):
        for h in range(p.Hkv):
            k, v = p.rows(s, h)
            o, pr, _, mags = attend(q[s, h * G:(h + 1) * G].double().numpy(), k, v, scale)
            got = out[s, h * G:(h + 1) * G]
            if L == 0:
                assert np.all(got == 0)
            else:
                assert np.all(np.abs(got - o) <= output_tolerance(pr, v, o, mags, p.D)), (s, h, np.abs(got - o).max())


def _call(pa, p, q, groups, scale, shared=None, ws=None, stream=None, max_shared=None, out=None):
    """groups: list of (rows, shared tokens)."""
    k, v, tables, ctx = p.cuda()
    rows = [r for g, _ in groups for r in g]
    starts = np.cumsum([0] + [len(g) for g, _ in groups])
    lens = [n for _, n in groups]
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    pa.pa_decode_shared(out, q.cuda(), k, v, tables, ctx, _i32(rows), _i32(starts), _i32(lens), max(p.lens),
                        max([0] + lens) if max_shared is None else max_shared, scale, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    return out


def _batch(Hkv, G, D, B, seed, groups, singles):
    """groups: (members, shared blocks, own lengths); singles: contexts.  Rows in a random order."""
    lens, lead = [], []
    for g, (m, nb, own) in enumerate(groups):
        for i in range(m):
            lens.append(nb * B + own[i % len(own)])
            lead.append((g, nb * B) if nb else None)
    lens += singles
    lead += [None] * len(singles)
    order = np.random.default_rng(seed).permutation(len(lens))
    p = Paged([lens[i] for i in order], Hkv, B, D, torch.bfloat16, seed, lead=[lead[i] for i in order])
    at = np.argsort(order)
    base, listed = 0, []
    for m, nb, _ in groups:
        listed.append(([int(at[base + i]) for i in range(m)], nb * B))
        base += m
    return p, p.q(len(lens), Hkv * G), listed


@pytest.mark.parametrize("Hkv,G,D,B", [(2, 1, 128, 16), (1, 2, 64, 32), (2, 4, 128, 16), (1, 8, 128, 32),
                                       (3, 1, 64, 16), (2, 4, 64, 32), (1, 8, 64, 16), (1, 2, 128, 32)])
def test_shared_against_the_definition(pa, Hkv, G, D, B):
    p, q, groups = _batch(Hkv, G, D, B, seed=G * D + B, groups=[
        (4, 3, [1, 17, 40]), (2, 1, [0, 5]), (1, 2, [9]), (130 // G, 5, [1, 2, 3, B, 600]), (3, 0, [7]), (3, 20, [0])],
        singles=[0, 1, 33, 700])
    out = _call(pa, p, q, groups, D ** -0.5)
    assert pa.pa_device_status() == 0
    _check(p, q, out, D ** -0.5, G)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1.5])
def test_shared_scales(pa, scale):
    p, q, groups = _batch(2, 2, 128, 16, seed=3, groups=[(5, 40, [1, 100]), (3, 9, [33])], singles=[50])
    ramp = torch.linspace(0.1, 3.0, p.width)
    done = set()
    for s, L in enumerate(p.lens):
        for i in range(-(-L // 16)):
            if p.tables[s, i] not in done:
                p.k[p.tables[s, i]] *= ramp[i]
                done.add(p.tables[s, i])
    out = _call(pa, p, q, groups, scale)
    assert pa.pa_device_status() == 0
    _check(p, q, out, scale, 2)


def test_shared_long_document_in_chunks(pa):
    p, q, groups = _batch(1, 4, 128, 32, seed=4, groups=[(40, 400, [1, 50, 900]), (2, 3, [2000])], singles=[9000, 17])
    out = _call(pa, p, q, groups, 0.09)
    assert pa.pa_device_status() == 0
    _check(p, q, out, 0.09, 4)


def test_shared_without_groups_is_plain_decode(pa):
    p, q, _ = _batch(2, 4, 128, 16, seed=5, groups=[], singles=[0, 1, 100, 512, 513, 1400, 16])
    k, v, tables, ctx = p.cuda()
    plain = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    pa.pa_decode(plain, q.cuda(), k, v, tables, ctx, 1400, 0.1)
    for groups in ([], [([1, 2], 0)]):
        out = _call(pa, p, q, groups, 0.1)
        assert pa.pa_device_status() == 0
        _check(p, q, out, 0.1, 4)
        # both keep 16 bits of a weight: they differ by the output's rounding, one step of bf16
        assert float((out.float() - plain.float()).abs().max()) <= 2.0 ** -7 * float(plain.float().abs().max())


def test_shared_very_long_own_tokens(pa):
    """More partitions of own tokens than a warp has lanes (contexts past 32 x 4096 tokens), beside a short group."""
    p, q, groups = _batch(1, 2, 64, 32, seed=11, groups=[(3, 4, [1, 30])], singles=[140001])
    out = _call(pa, p, q, groups, 0.125)
    assert pa.pa_device_status() == 0
    _check(p, q, out, 0.125, 2)


def test_shared_more_rows_than_a_plan_thread_each(pa):
    """Over 1024 rows: the plan keeps its per-row values in the workspace."""
    rng = np.random.default_rng(12)
    groups = [(int(m), int(nb), [int(x) for x in rng.integers(0, 30, 3)])
              for m, nb in zip(rng.integers(2, 6, 300), rng.integers(1, 4, 300))]
    p, q, listed = _batch(1, 1, 64, 16, seed=13, groups=groups, singles=[3, 600] * 60)
    assert len(p.lens) > 1024
    out = _call(pa, p, q, listed, 0.125)
    assert pa.pa_device_status() == 0
    _check(p, q, out, 0.125, 1)


def test_shared_many_small_groups(pa):
    rng = np.random.default_rng(6)
    groups = [(int(m), int(nb), [int(x) for x in rng.integers(0, 60, 3)])
              for m, nb in zip(rng.integers(2, 6, 250), rng.integers(1, 5, 250))]
    p, q, listed = _batch(2, 2, 64, 16, seed=7, groups=groups, singles=[5] * 40)
    out = _call(pa, p, q, listed, 0.125)
    assert pa.pa_device_status() == 0
    _check(p, q, out, 0.125, 2)


def test_shared_captured_beside_another_workspace_user(pa):
    p, q, groups = _batch(2, 4, 128, 16, seed=8, groups=[(9, 30, [1, 200]), (4, 7, [33])], singles=[800])
    first = _call(pa, p, q, groups, 0.1)
    k, v, tables, ctx = p.cuda()
    rows, starts = _i32([r for g, _ in groups for r in g]), _i32(np.cumsum([0] + [len(g) for g, _ in groups]))
    lens, qd, S = _i32([n for _, n in groups]), q.cuda(), len(p.lens)
    ws = torch.full((pa.pa_decode_shared_workspace_size(S, 8, 2, 128, 16, max(p.lens), 480, 2, 13),), 255,
                    dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(qd) for _ in range(2)]
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            pa.pa_decode_shared(o, qd, k, v, tables, ctx, rows, starts, lens, max(p.lens), 480, 0.1, workspace=ws,
                                stream=side)
        graphs.append(g)
    for _ in range(5):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert pa.pa_device_status() == 0
    for o in outs:
        assert np.array_equal(bits(o), bits(first))


def test_shared_back_to_back_calls_keep_their_order(pa):
    """Calls on one stream and one workspace, without waiting in between: each reads what the call before it wrote
    (the queries are the last output)."""
    p, q, groups = _batch(1, 2, 64, 16, seed=9, groups=[(12, 20, [1, 60])], singles=[300])
    k, v, tables, ctx = p.cuda()
    rows, starts, lens = _i32(groups[0][0]), _i32([0, 12]), _i32([320])
    ws = torch.empty(pa.pa_decode_shared_workspace_size(13, 2, 1, 64, 16, max(p.lens), 320, 1, 12), dtype=torch.uint8,
                     device="cuda")

    def chain(wait):
        x = q.cuda()
        for _ in range(20):
            y = torch.empty_like(x)
            pa.pa_decode_shared(y, x, k, v, tables, ctx, rows, starts, lens, max(p.lens), 320, 1.0, workspace=ws)
            if wait:
                torch.cuda.synchronize()
            x = y
        torch.cuda.synchronize()
        return x
    assert torch.equal(chain(True), chain(False))
    assert pa.pa_device_status() == 0


def test_shared_bad_groups_are_flagged_and_attend_on_their_own(pa):
    p, q, groups = _batch(1, 2, 128, 16, seed=10, groups=[(4, 6, [1, 30]), (3, 4, [20])], singles=[100])
    (r0, n0), (r1, n1) = groups
    S = len(p.lens)
    k, v, tables, ctx = p.cuda()
    cases = [
        ([r0, r1], [0, 4, 7], [n0 + 1, n1]),             # not whole blocks
        ([r0, r1], [0, 4, 7], [n0, 16 * 50]),            # longer than max_shared_len
        ([r0, r1], [0, 4, 7], [-16, n1]),
        ([r0, r1], [0, 4, 7], [112, n1]),                # longer than a member's context (97 tokens)
        ([r0, [S, r1[1], r1[2]]], [0, 4, 7], [n0, n1]),  # rows out of range
        ([r0, [-1, r1[1], r1[2]]], [0, 4, 7], [n0, n1]),
        ([r0, [r0[0], r1[1], r1[2]]], [0, 4, 7], [n0, n1]),   # a row listed twice
        ([r0, r1], [0, 5, 4], [n0, n1]),                 # starts that run backwards, or leave the rows
        ([r0, r1], [0, 4, 8], [n0, n1]),
        ([r0, r1], [-1, 4, 7], [n0, n1]),
    ]
    for rows, starts, lens in cases:
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        pa.pa_decode_shared(out, q.cuda(), k, v, tables, ctx, _i32(sum(rows, [])), _i32(starts), _i32(lens), max(p.lens),
                            112, 0.1)
        torch.cuda.synchronize()
        assert pa.pa_device_status() == pa.PA_DEV_BAD_CONTEXT, (starts, lens)
        _check(p, q, out, 0.1, 2)


@pytest.mark.parametrize("wid,over", [
    (6, dict(num_prompts=3, requests_per_prompt=5, stem_lens=(20, 150), suffix_lens=(1, 40), num_blocks=400)),
    (4, dict(num_prompts=4, streams_per_prompt=3, prompt_lens=(30, 90), private_tokens=(1, 30), num_blocks=600)),
    (7, dict(num_requests=3, beam_width=4, prompt_lens=(20, 90), beam_steps=9, num_blocks=400)),
    (3, dict(num_seqs=6, num_blocks=300, context_lens=[1, 15, 16, 17, 300, 77]))])
def test_batches_decode_shared(pa, wid, over):
    from paged_kv_cache_363_b200 import runner, workloads as W
    wl = W.make_workload(wid, seed=2, **over)
    b = runner.make_batch(wl, "cuda")
    b.append()
    plain = b.decode(out=torch.empty_like(b.out)).float()
    shared = b.decode_shared(out=torch.empty_like(b.out)).float()
    torch.cuda.synchronize()
    assert pa.pa_device_status() == 0
    (rows, starts, lens), longest = b.shared_groups()
    if wid != 3:
        assert rows.numel() > 0 and longest > 0
    # each side is within a weight's rounding of the definition; values of V are below 6
    assert float((plain - shared).abs().max()) <= 6 * 2.0 ** -8 + 2 * 2.0 ** -8 * float(plain.abs().max())


def test_shared_bad_group_beside_a_good_one(pa):
    """Contexts long enough that the good group's tokens are read once for all its rows."""
    p, q, groups = _batch(1, 2, 128, 16, seed=30, groups=[(4, 16, [1, 30]), (3, 14, [20])], singles=[300])
    (r0, n0), (r1, n1) = groups
    S = len(p.lens)
    for rows, starts, lens in (
            ([r0, r1], [0, 4, 7], [n0 + 1, n1]), ([r0, r1], [0, 4, 7], [n0, 16 * 50]), ([r0, r1], [0, 4, 7], [-16, n1]),
            ([r0, [S, r1[1], r1[2]]], [0, 4, 7], [n0, n1]), ([r0, [r0[0], r1[1], r1[2]]], [0, 4, 7], [n0, n1]),
            ([r0, r1], [0, 5, 4], [n0, n1])):
        k, v, tables, ctx = p.cuda()
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        pa.pa_decode_shared(out, q.cuda(), k, v, tables, ctx, _i32(sum(rows, [])), _i32(starts), _i32(lens), max(p.lens),
                            304, 0.1)
        torch.cuda.synchronize()
        assert pa.pa_device_status() == pa.PA_DEV_BAD_CONTEXT, (starts, lens)
        _check(p, q, out, 0.1, 2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("single", [1, 192, 193])
def test_shared_brief_contexts(pa, D, single):
    """Contexts of up to 192 tokens are read per row, longer ones once per group."""
    p, q, groups = _batch(2, 4, D, 16, seed=31 + single, groups=[(4, 5, [1, 17, 40]), (9, 8, [0, 64]), (2, 12, [0])],
                          singles=[single, 0])
    assert max(p.lens) == max(single, 192)
    out = _call(pa, p, q, groups, D ** -0.5)
    assert pa.pa_device_status() == 0
    _check(p, q, out, D ** -0.5, 4)
