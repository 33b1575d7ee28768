"""Blocks of the prefix cache that are unreferenced above a referenced one (CPU only): pa_alloc_make_private leaves them, and
nothing may count on evicting them."""
import numpy as np
import pytest

from oracle.allocator import OracleAllocator, OutOfBlocks as OracleOOM

pa = pytest.importorskip("paged_kv_cache_363_b200.pa", reason="libpa.so not built")


def _same(lib_a, ora, NB):
    assert lib_a.num_free() == ora.num_free() and lib_a.num_cached_free() == ora.num_cached_free()
    assert [lib_a.ref_count(b) for b in range(NB)] == ora.ref
    assert lib_a.stats()["num_seqs"] == len(ora.tables)
    for s in ora.tables:
        assert lib_a.num_tokens(s) == ora.ntokens[s]
        assert lib_a.block_table(s) == ora.tables[s]


def _pair(NB, B, order=None):
    return [pa.Allocator(NB, B, order), OracleAllocator(NB, B, order)]


def test_an_unreferenced_block_above_a_referenced_one_is_not_available():
    for a, oom in zip(_pair(4, 4), (pa.OutOfBlocks, OracleOOM)):
        a.add_seq_cached(0, list(range(12)))
        assert len(a.make_private(0, 4)) == 1       # the prompt's first block is released, its second one is not
        assert a.num_free() == 0 and a.num_cached_free() == 1
        with pytest.raises(oom):
            a.add_seq(1, 4)
        with pytest.raises(oom):
            a.add_seq_cached(1, list(range(100, 104)))
        _, cached = a.add_seq_cached(2, list(range(4)))
        assert cached == 4                          # its prompt can still be shared
        a.free_seq(2)
        a.truncate(0, 4)                            # lets go of the blocks behind the private one
        assert len(a.add_seq(1, 12)) == 12          # all three are evicted, leaf by leaf


def test_eviction_of_two_sequences_on_a_full_pool():
    for a, oom in zip(_pair(9, 4), (pa.OutOfBlocks, OracleOOM)):
        a.add_seq_cached(0, list(range(12)) + [1])
        a.add_seq_cached(1, list(range(12)) + [2])  # the same prompt: 3 shared blocks, 2 own ones, 4 free
        assert len(a.make_private(0, 8)) == 2
        assert len(a.make_private(1, 8)) == 2       # the shared two are unreferenced now, the third is not
        assert a.num_free() == 0 and a.num_cached_free() == 2
        with pytest.raises(oom):
            a.add_seq(2, 1)
        a.truncate(0, 8)
        a.truncate(1, 8)
        assert len(a.add_seq(2, 20)) == 20          # two own blocks, and the three of the cache


def test_beam_step_does_not_count_on_held_blocks():
    """An old beam that is dropped lets go of cached blocks that another sequence holds from below."""
    for a, oom in zip(_pair(6, 4), (pa.OutOfBlocks, OracleOOM)):
        a.add_seq_cached(0, list(range(12)))
        a.add_seq_cached(1, list(range(8)))          # an old beam on the first two blocks
        assert len(a.make_private(0, 8)) == 2        # sequence 0 keeps the third
        a.add_seq(2, 4)                              # another old beam; nothing is left
        assert a.num_free() == 0 and a.num_cached_free() == 0
        with pytest.raises(oom):
            a.beam_step([1, 2], [1], [3])            # two blocks lose their last reference, and can not be evicted
        assert a.num_tokens(1) == 8 if hasattr(a, "num_tokens") else a.ntokens[1] == 8
        a.truncate(0, 8)
        assert len(a.beam_step([1, 2], [1], [3])) > 0


def test_random_scripts_on_tight_pools():
    reached = sum(_random_script(seed) for seed in range(100))
    assert reached >= 10                             # scripts in which unreferenced blocks were held


def _random_script(seed):
    rng = np.random.default_rng(1000 + seed)
    NB, B = int(rng.integers(6, 26)), int(rng.choice([1, 2, 4]))
    order = rng.permutation(NB).astype(np.int32)
    lib_a, ora = _pair(NB, B, order)
    lib_a.add_host_pool(NB)
    ora.add_host_pool(NB)
    stems = [rng.integers(0, 2, size=8 * B).tolist() for _ in range(2)]
    nid, held = 0, False
    for _ in range(250):
        live = [s for s in ora.tables if s not in ora.on_host]
        kind = rng.choice(["add", "cached", "cached", "cached", "fork", "append", "free", "private", "private", "cut", "swap",
                           "beam"])
        s = int(rng.choice(live)) if live else None
        if kind == "add":
            args = (nid, int(rng.integers(0, 2 * B + 1)))
            name = "add_seq"
        elif kind == "cached":
            args, name = (nid, stems[rng.integers(2)][:int(rng.integers(1, 8 * B))]), "add_seq_cached"
        elif kind == "swap" and ora.on_host and rng.random() < 0.7:
            args, name = (int(rng.choice(sorted(ora.on_host))),), "swap_in"
        elif s is None:
            continue
        elif kind == "fork":
            args, name = (s, nid), "fork"
        elif kind == "beam":
            old = [int(x) for x in rng.permutation(live)[:int(rng.integers(1, 4))]]
            n = int(rng.integers(0, 4))
            args, name = (old, [int(x) for x in rng.integers(0, len(old), n)], list(range(nid, nid + n))), "beam_step"
            nid += n
        elif kind in ("private", "cut"):
            args = (s, int(rng.integers(0, ora.ntokens[s] + 1)))
            name = "make_private" if kind == "private" else "truncate"
        else:
            args, name = (s,), {"append": "append_slot", "free": "free_seq", "swap": "swap_out"}[kind]
        nid += 1
        try:
            want = getattr(ora, name)(*args)
        except OracleOOM:
            with pytest.raises(pa.OutOfBlocks):
                getattr(lib_a, name)(*args)
        except ValueError:
            with pytest.raises(pa.PAError):
                getattr(lib_a, name)(*args)
        else:
            got = getattr(lib_a, name)(*args)
            if name == "make_private":
                assert [tuple(x) for x in got.tolist()] == want
        held |= len(ora._evictable()) < ora.num_cached_free()
        _same(lib_a, ora, NB)
    for s in list(ora.tables):
        ora.free_seq(s)
        lib_a.free_seq(s)
    _same(lib_a, ora, NB)
    assert ora.available() == NB
    assert len(lib_a.add_seq(nid, NB * B)) == NB * B     # every block can be had again
    return held
