"""Groups of rows for pa_decode_shared that may nest (CPU only): against every way to group a small batch, and a recursion over
the prefix tree for larger ones."""
import os
import subprocess
import sys
import time

import numpy as np
import pytest

pa = pytest.importorskip("paged_kv_cache_363_b200.pa", reason="libpa.so not built")


def _partitions(items):
    if not items:
        yield []
        return
    for rest in _partitions(items[1:]):
        yield [[items[0]]] + rest
        for i in range(len(rest)):
            yield rest[:i] + [[items[0]] + rest[i]] + rest[i + 1:]


def _common(tables):
    d = 0
    while all(len(t) > d and t[d] == tables[0][d] for t in tables):
        d += 1
    return d


def _best_of_all(tables):
    """Every partition of the rows: a part saves its shared blocks once per row but the first."""
    return max(sum((len(p) - 1) * _common([tables[i] for i in p]) for p in parts)
               for parts in _partitions(list(range(len(tables)))))


def _best_over_tree(tables):
    """The same by recursion: every prefix has a group or has none, and a row is in the nearest one above it."""
    memo = {}

    def best(rows, depth, nearest):
        if len(rows) < 2:
            return nearest * len(rows)
        if (rows, nearest) not in memo:
            d = depth + _common([tables[i][depth:] for i in rows])

            def below(near):
                parts = {}
                for i in rows:
                    parts.setdefault(tables[i][d] if len(tables[i]) > d else None, []).append(i)
                ended = len(parts.pop(None, []))
                return near * ended + sum(best(tuple(p), d, near) for p in parts.values())
            memo[rows, nearest] = max(below(nearest), below(d) - d)
        return memo[rows, nearest]
    return best(tuple(range(len(tables))), 0, 0)


def _saved(a, ids, call):
    rows, starts, lens = call(ids)
    B = a.block_size
    full = [a.block_table(int(s))[:a.num_tokens(int(s)) // B] for s in ids]
    assert len(set(rows.tolist())) == len(rows) and starts[0] == 0 and starts[-1] == len(rows)
    saved, firsts = 0, []
    for g, L in enumerate(lens):
        r = rows[starts[g]:starts[g + 1]].tolist()
        assert len(r) >= 2 and L > 0 and L % B == 0 and r == sorted(r)
        assert len({tuple(full[i][:L // B]) for i in r}) == 1 and all(len(full[i]) >= L // B for i in r)
        saved += (len(r) - 1) * (L // B)
        firsts.append(r[0])
    assert firsts == sorted(firsts)
    return saved, full


def _prompts(rng, n, depth, kinds):
    """Token ids of n prompts (blocks of one token), each a walk down a random tree from a random point of the last."""
    out = [rng.integers(0, kinds, size=int(rng.integers(1, depth))).tolist()]
    for _ in range(n - 1):
        t = out[rng.integers(len(out))]
        out.append(t[:int(rng.integers(0, len(t) + 1))] + rng.integers(0, kinds, size=int(rng.integers(0, depth))).tolist())
    return out


@pytest.mark.parametrize("seed", range(60))
def test_small_batches_against_every_grouping(seed):
    rng = np.random.default_rng(seed)
    a = pa.Allocator(400, 1)
    n = int(rng.integers(2, 8))
    for i, t in enumerate(_prompts(rng, n, int(rng.integers(2, 12)), 2)):
        a.add_seq_cached(i, t)
    ids = rng.permutation(n)
    saved, full = _saved(a, ids, a.nested_groups)
    assert saved == _best_of_all(full) == _best_over_tree(full)
    assert saved >= _saved(a, ids, a.shared_groups)[0]


@pytest.mark.parametrize("seed", range(60))
def test_larger_batches_against_the_tree(seed):
    rng = np.random.default_rng(100 + seed)
    B = int(rng.choice([1, 2, 4]))
    a = pa.Allocator(20000, B, rng.permutation(20000).astype(np.int32))
    n = int(rng.integers(10, 90))
    for i, t in enumerate(_prompts(rng, n, int(rng.integers(2, 40)), int(rng.integers(2, 4)))):
        kind = rng.integers(5)
        if kind == 0 and i:
            a.fork(int(rng.integers(i)), i)
        elif kind == 1:
            a.add_seq(i, int(rng.integers(0, 9)))
        else:
            a.add_seq_cached(i, np.repeat(t, B).tolist() + [7] * int(rng.integers(0, B)))
    ids = rng.permutation(n)[:max(1, n - 3)]
    saved, full = _saved(a, ids, a.nested_groups)
    assert saved == _best_over_tree(full)
    assert saved >= _saved(a, ids, a.shared_groups)[0]


def test_two_long_documents_behind_a_stem_of_a_hundred():
    a = pa.Allocator(7000, 16)
    stem, document = list(range(64 * 16)), [5] * (6400 * 16)
    for i in range(100):
        a.add_seq_cached(i, (stem + document if i in (3, 70) else stem) + [100000 + i])
    rows, starts, lens = a.nested_groups(np.arange(100))
    assert starts.tolist() == [0, 98, 100] and lens.tolist() == [64 * 16, 6464 * 16]
    assert rows[98:].tolist() == [3, 70] and sorted(rows.tolist()) == list(range(100))
    # without nesting: the two alone, or all by the stem alone
    rows, starts, lens = a.shared_groups(np.arange(100))
    assert (rows.tolist(), lens.tolist()) in (([3, 70], [6464 * 16]), (list(range(100)), [64 * 16]))


def test_none_and_refusals():
    a = pa.Allocator(8, 4)
    rows, starts, lens = a.nested_groups([])
    assert (len(rows), starts.tolist(), len(lens)) == (0, [0], 0)
    a.add_host_pool(4)
    a.add_seq(0, 8)
    a.fork(0, 1)
    assert a.nested_groups([1, 0])[2].tolist() == [8]
    a.swap_out(1)
    for ids in ([1, 0], [5]):
        with pytest.raises(pa.PAError):
            a.nested_groups(ids)


def test_deep_nesting_in_time():
    """Every row shares one block more with the next than with the one before."""
    a = pa.Allocator(400, 1)
    for i in range(150):
        a.add_seq_cached(i, [0] * i + [i + 1])
    saved, full = _saved(a, np.arange(150), a.nested_groups)
    assert saved == _best_over_tree(full)
    n = 1500
    a = pa.Allocator(3 * n, 1)
    for i in range(n):
        a.add_seq_cached(i, [0] * i + [i + 1])
    t0 = time.perf_counter()
    rows, starts, lens = a.nested_groups(np.arange(n))
    assert time.perf_counter() - t0 < 20
    saved, _ = _saved(a, np.arange(n), a.nested_groups)
    assert saved >= _saved(a, np.arange(n), a.shared_groups)[0] > 0
    assert len(lens) > 1


@pytest.mark.parametrize("call", ["shared_groups", "nested_groups"])
def test_without_host_memory_the_call_fails(call):
    """A batch whose lists do not fit in the process's address space: an error, and the process lives on."""
    program = """
import resource
import numpy as np
from paged_kv_cache_363_b200 import pa
a = pa.Allocator(4, 4)
a.add_seq(0, 4)
ids = np.zeros(60_000_000, np.int64)
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + 900_000_000, used + 900_000_000))  # room for the 480 MB of results alone
try:
    a.%s(ids)
except pa.PAError as e:
    assert "host allocation failed" in str(e), e
    print("refused")
assert a.num_tokens(0) == 4
""" % call
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", program], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr
