"""Host side of the operators beside plain decode and prefill (CPU only): argument checks of the
C ABI and the binding, workspace sizes, and the allocator calls that go with them."""
import ctypes

import numpy as np
import pytest

from oracle.allocator import OracleAllocator, OutOfBlocks as OracleOOM

pa = pytest.importorskip("paged_kv_cache_363_b200.pa", reason="libpa.so not built")

P = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1008)


def _scores(out=P, scores=P, q=P, S=1, Hq=4, Hkv=4, D=128, B=16, ctx=64, stride=64, scale=1.0, part=0, ws=P, nbytes=1 << 30,
            dt=1):
    return pa.lib.pa_decode_scores(out, scores, q, P, P, P, P, S, Hq, Hkv, D, B, 4, 8, ctx, stride, scale, part, ws, nbytes,
                                   dt, None)


@pytest.mark.parametrize("bad,code", [
    (dict(D=96), "UNSUPPORTED"), (dict(B=8), "UNSUPPORTED"), (dict(dt=7), "UNSUPPORTED"), (dict(Hq=12), "UNSUPPORTED"),
    (dict(Hq=6), "INVALID"), (dict(stride=63), "INVALID"), (dict(scores=None), "INVALID"), (dict(q=ODD), "INVALID"),
    (dict(scale=float("nan")), "INVALID"), (dict(part=24), "INVALID"), (dict(ws=None), "INVALID"),
    (dict(nbytes=64), "INVALID"), (dict(S=65536), "INVALID"), (dict(ctx=-1), "INVALID")])
def test_decode_scores_refusals(bad, code):
    assert _scores(**bad) == getattr(pa, "PA_ERR_" + code)
    assert "pa_decode_scores" in pa.lib.pa_last_error_string().decode() or "partition" in \
        pa.lib.pa_last_error_string().decode()


def test_decode_scores_without_sequences_and_workspace():
    assert _scores(S=0, out=None, scores=None, ws=None, nbytes=0) == pa.PA_OK
    plain = pa.pa_decode_workspace_size(8, 32, 8, 128, 16, 1000)
    assert pa.pa_decode_scores_workspace_size(8, 32, 8, 128, 16, 1000) >= plain + 4 * 8 * 32 * 1000
    assert pa.pa_decode_scores_workspace_size(0, 32, 8, 128, 16, 1000) == 0


def _evict(k=P, ns=P, recent=0, S=1, Hkv=4, D=128, B=16, ctx=64, stride=64, ws=P, nbytes=1 << 30, dt=1):
    return pa.lib.pa_evict(k, P, ns, P, P, P, P, P, P, recent, S, Hkv, D, B, 4, 8, ctx, stride, ws, nbytes, dt, None)


@pytest.mark.parametrize("bad,code", [
    (dict(D=96), "UNSUPPORTED"), (dict(B=8), "UNSUPPORTED"), (dict(dt=7), "UNSUPPORTED"), (dict(Hkv=0), "INVALID"),
    (dict(recent=-1), "INVALID"), (dict(stride=63), "INVALID"), (dict(k=None), "INVALID"), (dict(k=ODD), "INVALID"),
    (dict(ns=None), "INVALID"), (dict(ws=None), "INVALID"), (dict(nbytes=8), "INVALID"), (dict(S=-1), "INVALID"),
    (dict(ctx=262145, stride=262145), "UNSUPPORTED"), (dict(S=65535, Hkv=17), "UNSUPPORTED")])
def test_evict_refusals(bad, code):
    assert _evict(**bad) == getattr(pa, "PA_ERR_" + code)
    assert "pa_evict" in pa.lib.pa_last_error_string().decode()


def test_evict_nothing_to_do_and_workspace():
    assert _evict(S=0, k=None, ws=None) == pa.PA_OK
    assert _evict(ctx=0, k=None, ws=None) == pa.PA_OK
    # a move has a slot on either side of the budget: at most half the context, 8 bytes each, and a count
    assert pa.pa_evict_workspace_size(3, 4, 101) >= 3 * 4 * (8 * 50 + 4)
    assert pa.pa_evict_workspace_size(3, 4, 262145) == 0
    assert pa.pa_evict_workspace_size(0, 4, 10) == 0


def _cross(out=P, lse=None, q=P, S=1, Hq=4, Hkv=4, D=128, B=16, mb=4, NB=8, Nq=5, mq=5, ctx=64, scale=1.0, ws=P,
           nbytes=1 << 30, dt=1):
    return pa.lib.pa_cross_attention(out, lse, q, P, P, P, P, P, S, Hq, Hkv, D, B, mb, NB, Nq, mq, ctx, scale, ws, nbytes, dt,
                                     None)


@pytest.mark.parametrize("bad,code", [
    (dict(D=96), "UNSUPPORTED"), (dict(B=8), "UNSUPPORTED"), (dict(dt=0), "UNSUPPORTED"), (dict(Hq=12), "UNSUPPORTED"),
    (dict(Hq=6), "INVALID"), (dict(Hq=0), "INVALID"), (dict(q=ODD), "INVALID"), (dict(out=None), "INVALID"),
    (dict(lse=ctypes.c_void_p(0x1002)), "INVALID"), (dict(scale=float("inf")), "INVALID"), (dict(ws=None), "INVALID"),
    (dict(nbytes=64), "INVALID"), (dict(S=65536), "INVALID"), (dict(ctx=-1), "INVALID"), (dict(mq=-1), "INVALID"),
    (dict(NB=1 << 26), "UNSUPPORTED"), (dict(Nq=2 ** 31 - 1, Hq=128, Hkv=16), "UNSUPPORTED")])
def test_cross_attention_refusals(bad, code):
    assert _cross(**bad) == getattr(pa, "PA_ERR_" + code)
    assert "pa_cross_attention" in pa.lib.pa_last_error_string().decode()


def test_cross_attention_nothing_to_do_and_workspace():
    for none in (dict(S=0), dict(Nq=0), dict(mq=0)):
        assert _cross(out=None, q=None, ws=None, **none) == pa.PA_OK
    # without partial states: entries alone; with few rows and a long context, 32 states per (row, head) at most
    many = pa.pa_cross_attention_workspace_size(4, 32, 8, 128, 16, 100000, 50000, 1 << 20)
    assert 0 < many < 100000 * 32
    few = pa.pa_cross_attention_workspace_size(1, 8, 1, 128, 16, 1, 1, 1 << 20)
    assert 32 * 8 * (128 + 2) * 4 <= few <= 2 * 32 * 8 * (128 + 2) * 4
    assert pa.pa_cross_attention_workspace_size(1, 12, 4, 128, 16, 1, 1, 64) == 0


def _shared(out=P, q=P, rows=P, start=P, lens=P, S=8, Hq=4, Hkv=4, D=128, B=16, mb=4, NB=8, ng=2, nr=6, ctx=64, sh=32,
            scale=1.0, ws=P, nbytes=1 << 30, dt=1):
    return pa.lib.pa_decode_shared(out, q, P, P, P, P, rows, start, lens, S, Hq, Hkv, D, B, mb, NB, ng, nr, ctx, sh, scale, ws,
                                   nbytes, dt, None)


@pytest.mark.parametrize("bad,code", [
    (dict(D=96), "UNSUPPORTED"), (dict(B=8), "UNSUPPORTED"), (dict(dt=0), "UNSUPPORTED"), (dict(Hq=12), "UNSUPPORTED"),
    (dict(Hq=6), "INVALID"), (dict(nr=9), "INVALID"), (dict(ng=-1), "INVALID"), (dict(sh=-1), "INVALID"),
    (dict(rows=None), "INVALID"), (dict(start=None), "INVALID"), (dict(lens=None), "INVALID"), (dict(q=ODD), "INVALID"),
    (dict(scale=float("nan")), "INVALID"), (dict(ws=None), "INVALID"), (dict(nbytes=64), "INVALID"),
    (dict(S=65536), "INVALID"), (dict(mb=0), "INVALID"), (dict(NB=1 << 26), "UNSUPPORTED")])
def test_decode_shared_refusals(bad, code):
    assert _shared(**bad) == getattr(pa, "PA_ERR_" + code)
    assert "pa_decode_shared" in pa.lib.pa_last_error_string().decode()


def test_decode_shared_nothing_to_do_and_workspace():
    assert _shared(S=0, nr=0, out=None, q=None, ws=None) == pa.PA_OK
    # a partial state per chunk and per partition, for every row and head; no groups need no chunks
    w = pa.pa_decode_shared_workspace_size(8, 32, 8, 128, 16, 1000, 512, 2, 8)
    assert w >= 8 * 32 * (2 + 2) * 130 * 4
    assert 0 < pa.pa_decode_shared_workspace_size(8, 32, 8, 128, 16, 1000, 0, 0, 0) < w
    assert pa.pa_decode_shared_workspace_size(8, 32, 8, 128, 16, 1000, -1, 0, 0) == 0


def _best_saving(tables):
    """The most block reads any grouping of rows by common leading blocks saves, by recursion over prefixes."""
    if len(tables) < 2:
        return 0
    d = 0
    while all(len(t) > d and t[d] == tables[0][d] for t in tables):
        d += 1
    parts = {}
    for t in tables:
        if len(t) > d:
            parts.setdefault(t[d], []).append(t)
    return max((len(tables) - 1) * d, sum(_best_saving(p) for p in parts.values()))


@pytest.mark.parametrize("seed", range(20))
def test_shared_groups_save_the_most(seed):
    rng = np.random.default_rng(seed)
    B = int(rng.choice([2, 4]))
    a = pa.Allocator(3000, B, rng.permutation(3000).astype(np.int32))
    stems = [rng.integers(0, 3, size=40).tolist() for _ in range(3)]
    n = int(rng.integers(1, 40))
    for i in range(n):
        kind = rng.integers(4)
        if kind == 0 or i == 0:
            a.add_seq(i, int(rng.integers(0, 5 * B)))
        elif kind == 1:
            a.fork(int(rng.integers(i)), i)
        else:
            s = stems[rng.integers(3)]
            a.add_seq_cached(i, s[:int(rng.integers(1, 40))] + rng.integers(3, 9, size=5).tolist())
        for _ in range(int(rng.integers(0, 4))):
            a.append_slot(i)
    ids = rng.permutation(n)[:max(1, n - 2)]
    rows, starts, lens = a.shared_groups(ids)
    full = [a.block_table(int(s))[:a.num_tokens(int(s)) // B] for s in ids]
    assert len(set(rows.tolist())) == len(rows) and starts[0] == 0 and starts[-1] == len(rows)
    saved, firsts = 0, []
    for g, L in enumerate(lens):
        r = rows[starts[g]:starts[g + 1]]
        assert len(r) >= 2 and L > 0 and L % B == 0 and r.tolist() == sorted(r.tolist())
        assert len({tuple(full[i][:L // B]) for i in r}) == 1 and all(len(full[i]) >= L // B for i in r)
        saved += (len(r) - 1) * (L // B)
        firsts.append(r[0])
    assert firsts == sorted(firsts)
    assert saved == _best_saving(full)


def test_shared_groups_of_none_and_of_swapped_sequences():
    a = pa.Allocator(8, 4)
    rows, starts, lens = a.shared_groups([])
    assert (len(rows), starts.tolist(), len(lens)) == (0, [0], 0)
    a.add_host_pool(4)
    a.add_seq(0, 8)
    a.fork(0, 1)
    assert a.shared_groups([1, 0])[2].tolist() == [8]
    a.swap_out(1)
    with pytest.raises(pa.PAError):
        a.shared_groups([1, 0])
    with pytest.raises(pa.PAError):
        a.shared_groups([5])


def _same(lib_a, ora, NB):
    assert lib_a.num_free() == ora.num_free() and lib_a.num_cached_free() == ora.num_cached_free()
    assert [lib_a.ref_count(b) for b in range(NB)] == ora.ref
    for s in ora.tables:
        assert lib_a.num_tokens(s) == ora.ntokens[s]
        assert lib_a.block_table(s) == ora.tables[s]
    assert lib_a.stats()["cow_copies"] == ora.cow_count


@pytest.mark.parametrize("seed", range(12))
def test_make_private_and_truncate_match_the_oracle(seed):
    rng = np.random.default_rng(seed)
    NB, B = int(rng.integers(12, 60)), int(rng.choice([2, 4, 16]))
    order = rng.permutation(NB).astype(np.int32)
    lib_a, ora = pa.Allocator(NB, B, order), OracleAllocator(NB, B, order)
    lib_a.add_host_pool(NB)
    ora.add_host_pool(NB)
    stems = [rng.integers(0, 3, size=6 * B).tolist() for _ in range(2)]
    nid, seen = 0, set()
    for _ in range(120):
        live = list(ora.tables)
        kind = rng.choice(["add", "cached", "fork", "append", "free", "private", "private", "cut", "cut", "swap"])
        s = int(rng.choice(live)) if live else None
        try:
            if kind == "add":
                args = (nid, int(rng.integers(0, 4 * B)))
                fo, fl = ora.add_seq, lib_a.add_seq
            elif kind == "cached":
                args = (nid, stems[rng.integers(2)][:int(rng.integers(1, 6 * B))])
                fo, fl = ora.add_seq_cached, lib_a.add_seq_cached
            elif s is None:
                continue
            elif kind == "fork":
                args, fo, fl = (s, nid), ora.fork, lib_a.fork
            elif kind == "append":
                args, fo, fl = (s,), ora.append_slot, lib_a.append_slot
            elif kind == "free":
                args, fo, fl = (s,), ora.free_seq, lib_a.free_seq
            elif kind == "swap":
                args, fo, fl = ((s,), ora.swap_in, lib_a.swap_in) if s in ora.on_host else \
                    ((s,), ora.swap_out, lib_a.swap_out)
            else:
                n = int(rng.integers(0, ora.ntokens[s] + 2))      # sometimes one more than it has
                args, fo, fl = ((s, n), ora.make_private, lib_a.make_private) if kind == "private" else \
                    ((s, n), ora.truncate, lib_a.truncate)
            nid += 1
            want = fo(*args)
        except OracleOOM:
            with pytest.raises(pa.OutOfBlocks):
                fl(*args)
            seen.add("oom " + kind)
        except ValueError:
            with pytest.raises(pa.PAError):
                fl(*args)
            seen.add("refused " + kind)
        else:
            got = fl(*args)
            if kind == "private":
                assert [tuple(x) for x in got.tolist()] == want
                assert len({d for _, d in want} & {x for x, _ in want}) == 0
                pa.pa_check_block_mapping(got, NB)
                seen.add("copied" if want else "none")
        _same(lib_a, ora, NB)
    assert "copied" in seen and "refused private" in seen and "refused cut" in seen


def test_truncate_keeps_cached_blocks_whole():
    a = pa.Allocator(8, 4)
    a.add_seq_cached(0, list(range(12)))
    with pytest.raises(pa.PAError):
        a.truncate(0, 6)                     # would leave a cached block as the partial last one
    a.truncate(0, 8)
    assert len(a.make_private(0, 6)) == 2
    a.truncate(0, 6)
    slot, cow = a.append_slot(0)
    assert cow is None and slot == a.block_table(0)[1] * 4 + 2
    _, cached = a.add_seq_cached(1, list(range(12)))
    assert cached == 12                      # the cache still holds the prompt's blocks
