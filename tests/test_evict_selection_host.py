"""pa_evict's selection on the host (CPU only): the passes over key ranges, run by a C++ program that includes the
kernel's own arithmetic, against a sort."""
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_363_b200", "csrc")

PROGRAM = r"""
#include "pa_evict_select.h"
extern "C" uint32_t score_key(float x) { return pa::score_key(x); }
// The threshold among L keys for the n best, and how many of its equals are among them; the number of passes, or
// -1 where no bin holds the n-th key.
extern "C" int select_keys(const uint32_t* range_keys, const uint32_t* keys, int L, uint32_t n, uint32_t few, uint32_t* prefix,
                           uint32_t* need)
{
    pa::KeyRange r{0xffffffffu, 0u};
    for (int i = 0; i < L; ++i) {                        // (of the scores: before the recent tokens are marked)
        if (range_keys[i] < r.lo) r.lo = range_keys[i];
        if (range_keys[i] > r.hi) r.hi = range_keys[i];
    }
    *prefix = pa::kRecentKey;
    *need = n;
    for (int pass = 0; pass < pa::kEvictPasses; ++pass) {
        const int shift = r.shift();
        static uint32_t hist[pa::kEvictBins];
        for (uint32_t& h : hist) h = 0;
        uint32_t recent = 0;
        for (int i = 0; i < L; ++i) {
            if (keys[i] == pa::kRecentKey) ++recent;
            if (!r.has(keys[i])) continue;
            const uint32_t b = r.bin(keys[i], shift);
            if (b >= (uint32_t)pa::kEvictBins) return -2;
            ++hist[b];
        }
        if (pass == 0) {
            if (recent >= *need) return pass + 1;
            *need -= recent;
        }
        int b = pa::kEvictBins - 1;
        uint32_t above = 0;
        while (b >= 0 && above + hist[b] < *need) above += hist[b--];
        if (b < 0) return -1;
        *prefix = r.first((uint32_t)b, shift);
        *need -= above;
        if (shift == 0) return pass + 1;
        r = r.narrow(*prefix, shift);
        if (r.lo > r.hi) return -3;
        if (hist[b] > few) continue;
        for (int i = 0; i < L; ++i) {                    // few left: each is compared with all
            if (!r.has(keys[i])) continue;
            uint32_t more = 0, same = 0;
            for (int j = 0; j < L; ++j) {
                if (!r.has(keys[j])) continue;
                more += keys[j] > keys[i];
                same += keys[j] == keys[i];
            }
            if (more < *need && *need <= more + same) {
                *prefix = keys[i];
                *need -= more;
                return pass + 1;
            }
        }
        return -1;
    }
    return -4;                                           // a fourth pass would be needed
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    import ctypes
    d = tmp_path_factory.mktemp("evict")
    src, lib = str(d / "select.cpp"), str(d / "select.so")
    with open(src, "w") as f:
        f.write(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib], check=True)
    h = ctypes.CDLL(lib)
    h.score_key.argtypes, h.score_key.restype = [ctypes.c_float], ctypes.c_uint32
    return h


def _key(x):
    b = (np.asarray(x, np.float32) + np.float32(0)).view(np.uint32)
    k = np.where(b >> 31, ~b, b | np.uint32(1 << 31))
    return np.where(np.isnan(x), np.uint32(0xfffffffe), k).astype(np.uint32)


def _check(host, score_keys, recent, n, few=256):
    keys = score_keys.copy()
    keys[recent] = 0xffffffff
    prefix, need = np.zeros(1, np.uint32), np.zeros(1, np.uint32)
    import ctypes
    ptr = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    passes = host.select_keys(ptr(score_keys), ptr(keys), len(keys), ctypes.c_uint32(n), ctypes.c_uint32(few), ptr(prefix),
                              ptr(need))
    want = np.sort(keys)[::-1][n - 1]
    assert 1 <= passes <= 3
    assert prefix[0] == want and need[0] == n - np.count_nonzero(keys > want)


def test_keys_in_the_order_of_scores(host):
    x = np.array([-np.inf, -3e38, -1.0, -1e-42, -0.0, 0.0, 1e-42, 1.0, 3e38, np.inf, np.nan, -np.nan], np.float32)
    k = [host.score_key(float(v)) for v in x]
    assert k == _key(x).tolist()
    assert k[4] == k[5] and k[-1] == k[-2] and sorted(set(k)) == list(dict.fromkeys(k))


@pytest.mark.parametrize("least", [1e-3, 0.1, 1.0, 0.0, -1e-6, -0.7, -np.inf, 1e30, np.inf])
@pytest.mark.parametrize("nans", [1, 20, 256, 257, 900, 1300])
def test_nan_among_scores(host, least, nans):
    """The top bin of a range that holds NaN may end past 2^32."""
    rng = np.random.default_rng(nans)
    L = 1400
    for recents in (0, 128):
        x = np.exp(rng.standard_normal(L)).astype(np.float32)
        x = np.maximum(x, np.float32(max(least, 0.0))) if least >= 0 else x
        x[rng.integers(L)] = least
        x[rng.permutation(L)[:nans]] = np.nan
        recent = rng.permutation(L)[:recents]
        for n in (1, 10, nans - 1, nans, nans + 1, nans + recents, nans + recents + 1, 1024, L - 1):
            if 0 < n < L:
                _check(host, _key(x), recent, n)


@pytest.mark.parametrize("few", [0, 1, 256])
def test_ranges_from_any_key_to_any_other(host, few):
    """Keys of any bits (NaN's among them or not), the smallest at an arbitrary odd one."""
    rng = np.random.default_rng(few)
    for trial in range(400):
        lo = int(rng.integers(0, 2 ** 32 - 1)) | 1
        hi = int(rng.choice([0xfffffffe, 0xff800000, rng.integers(0, 2 ** 32 - 1)]))
        lo, hi = min(lo, hi), max(lo, hi)
        L = int(rng.integers(2, 700))
        keys = rng.integers(lo, hi + 1, size=L).astype(np.uint32)
        if trial % 3 == 0:
            keys[rng.random(L) < 0.5] = hi
        elif trial % 3 == 1:
            keys = np.maximum(keys, np.uint32(max(lo, hi - 5000)))
        keys[0] = lo
        n = int(rng.integers(1, L))
        _check(host, keys, rng.permutation(L)[:int(rng.integers(0, 20))], n, few)
