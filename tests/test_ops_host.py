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
