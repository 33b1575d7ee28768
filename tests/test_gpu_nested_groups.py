"""pa_decode_shared of groups that nest, as pa_alloc_nested_groups finds them, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from pa_ops_testlib import Paged
from test_gpu_shared import _check, _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G,D,own", [(1, 64, 5), (4, 128, 300)])
def test_shared_nested_groups(G, D, own):
    from paged_kv_cache_363_b200 import pa
    B, Hkv = 16, 2
    a = pa.Allocator(600, B, np.random.default_rng(1).permutation(600).astype(np.int32))
    stem, document = list(range(7 * B)), [3] * (60 * B)
    for i in range(12):
        tail = list(range(1000 * (i + 1), 1000 * (i + 1) + (i * own) // 11 + 1))
        a.add_seq_cached(i, (stem + document if i in (2, 5, 9) else stem if i != 7 else []) + tail)
    rows, starts, lens = a.nested_groups(np.arange(12))
    assert sorted(lens.tolist()) == [7 * B, 67 * B] and len(rows) == 11
    tables, ctx = a.block_tables(np.arange(12), max(len(a.block_table(i)) for i in range(12)))
    p = Paged([1], Hkv, B, D, torch.bfloat16, seed=3)       # (its pools and tables are replaced)
    rng = np.random.default_rng(4)
    p.lens, p.tables = [int(x) for x in ctx], tables
    p.k, p.v = (torch.from_numpy(rng.standard_normal((600, Hkv, B, D), dtype=np.float32)).to(torch.bfloat16) for _ in range(2))
    q = p.q(12, Hkv * G)
    k, v, t, c = p.cuda()
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    pa.pa_decode_shared(out, q.cuda(), k, v, t, c, _i32(rows), _i32(starts), _i32(lens), max(p.lens), int(lens.max()), D ** -0.5)
    torch.cuda.synchronize()
    assert pa.pa_device_status() == 0
    _check(p, q, out, D ** -0.5, G)
