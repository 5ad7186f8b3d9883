"""qsvd_evict_rows against the definition: the kept rows, and every byte moved, exactly."""
import numpy as np
import pytest
import torch

import rank_joint_qkv_b200 as q
from tests.serving_util import DEV, keep_rows

pytestmark = pytest.mark.gpu
ROW = {"f32": 4, "f16": 2, "bf16": 2, "i8": 1, "i4": 0.5}


def setup(cache, r, group, max_len, lens, seed, dst_max_len=None):
    g = np.random.default_rng(seed)
    B, rb = len(lens), int(r * ROW[cache])
    dims = q.make_dims(64, 1, 64, r, B, max_len, cache=cache, group=group)
    rows = g.integers(0, 256, (B, max_len, rb), dtype=np.uint8)       # any bytes: rows are moved, not read
    ng = r // group if cache in ("i8", "i4") else 0
    scales = g.integers(0, 65536, (B, max_len, ng)).astype(np.uint16) if ng else None
    w = np.exp(2 * g.standard_normal((B, max_len))).astype(np.float32)
    w[g.random((B, max_len)) < 0.2] = 0.0                            # many equal weights
    w[g.random((B, max_len)) < 0.1] = np.float32(0.5)
    return dims, rows, scales, w


def to_dev(a):
    return None if a is None else torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).to(DEV)


def run_and_check(cache, r, group, max_len, lens, budget, sink, recent, in_place, seed=0, weights=None):
    dims, rows, scales, w = setup(cache, r, group, max_len, lens, seed)
    if weights is not None:
        w = weights
    B, L2 = len(lens), max_len if in_place else budget + 3
    d_rows, d_sc, d_w = to_dev(rows), to_dev(scales), to_dev(w)
    d_len = torch.tensor(lens, dtype=torch.int32, device=DEV)
    kept = torch.full((B, budget), 99, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    if in_place:
        q.qsvd_evict_rows(dims, d_w, d_len, budget, d_rows, d_sc, sink=sink, recent=recent, kept=kept, status=status)
        o_rows, o_sc, o_w, o_len = d_rows, d_sc, d_w, d_len
        left_rows, left_sc = rows, scales
    else:
        left_rows = np.full((B, L2, rows.shape[2]), 171, np.uint8)
        left_sc = None if scales is None else np.full((B, L2, scales.shape[2]), 43981, np.uint16)
        o_rows, o_sc = to_dev(left_rows), to_dev(left_sc)
        o_w = torch.full((B, L2), 5.0, device=DEV)
        o_len = torch.zeros(B, dtype=torch.int32, device=DEV)
        q.qsvd_evict_rows(dims, d_w, d_len, budget, d_rows, d_sc, sink=sink, recent=recent, dst_max_len=L2, dst_cache=o_rows,
                          dst_scales=o_sc, dst_weights=o_w, dst_lengths=o_len, kept=kept, status=status)
    torch.cuda.synchronize()
    o_rows, o_w, o_len, kept = (t.cpu().numpy() for t in (o_rows, o_w, o_len, kept))
    o_sc = None if o_sc is None else o_sc.cpu().numpy().view(np.uint16)
    flags = 0
    for b, n in enumerate(lens):
        if n < 0 or n > max_len:
            flags = q.QSVD_STATUS_LEN_CLAMPED
        n = min(max(n, 0), max_len)
        at = keep_rows(w[b, :n], n, budget, sink, recent)
        m = len(at)
        assert o_len[b] == m == min(n, budget)
        assert kept[b, :m].tolist() == at and (kept[b, m:] == -1).all()
        assert np.array_equal(o_rows[b, :m], rows[b, at])
        assert np.array_equal(o_rows[b, m:], left_rows[b, m:])          # rows behind are left as they were
        if scales is not None:
            assert np.array_equal(o_sc[b, :m], scales[b, at]) and np.array_equal(o_sc[b, m:], left_sc[b, m:])
        assert np.array_equal(o_w[b, :m].view(np.uint32), w[b, at].view(np.uint32))
        assert (o_w[b, m:] == 0).all()
    assert int(status.item()) == flags
    if not in_place:   # the sources are untouched
        assert np.array_equal(d_rows.cpu().numpy(), rows) and np.array_equal(d_w.cpu().numpy().view(np.uint32), w.view(np.uint32))


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("cache,r,group", [("f32", 32, 32), ("f16", 256, 128), ("bf16", 96, 32), ("i8", 256, 128),
                                           ("i8", 96, 32), ("i4", 32, 32), ("i4", 768, 128), ("f16", 1536, 128)])
def test_every_type(cuda_ok, cache, r, group, in_place):
    run_and_check(cache, r, group, 700, (0, 1, 63, 64, 65, 700, 333), 64, 4, 16, in_place)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("max_len,lens,budget,sink,recent", [
    (5, (5, 4, 0), 1, 0, 0),           # one row: the heaviest
    (5, (5, 3, 1), 1, 1, 0),           # ... the first
    (5, (5, 2, 5), 1, 0, 1),           # ... the last
    (40, (40, 33, 40), 32, 16, 16),    # nothing left for the weights
    (40, (40, 40), 40, 0, 0),          # the budget is the capacity
    (1500, (1500, 1024, 1025), 1024, 0, 0),
    (3001, (3001, 2047, 2049), 1999, 7, 500),
    (600, (600, -5, 4000), 100, 4, 10),   # lengths out of range are clamped and flagged
])
def test_budgets_and_lengths(cuda_ok, max_len, lens, budget, sink, recent, in_place):
    run_and_check("f16", 64, 32, max_len, lens, budget, sink, recent, in_place, seed=5)


@pytest.mark.parametrize("in_place", [True, False])
def test_long_sequence(cuda_ok, in_place):
    run_and_check("f16", 256, 128, 30011, (30011, 20000), 9001, 4, 1000, in_place, seed=7)
    run_and_check("i4", 128, 32, 70001, (70001,), 8192, 4, 128, in_place, seed=8)


def test_special_weights(cuda_ok):
    """Infinities, NaN of either sign, both zeros, the smallest and largest numbers, all equal, falling and rising."""
    n = 400
    g = np.random.default_rng(1)
    bad = np.array([np.inf, -np.inf, np.nan, -np.nan, 0.0, -0.0, 1e-45, -1e-45, 3.4e38, -3.4e38, 1.0], np.float32)
    w = np.stack([bad[g.integers(0, len(bad), n)], np.zeros(n, np.float32), np.full(n, np.nan, np.float32),
                  np.arange(n, 0, -1).astype(np.float32), np.arange(n).astype(np.float32),
                  np.where(np.arange(n) % 2 == 0, 0.0, -0.0).astype(np.float32)])
    for budget, sink, recent in ((150, 4, 16), (399, 0, 0), (1, 0, 0)):
        for in_place in (True, False):
            run_and_check("f16", 64, 32, n, (n,) * 6, budget, sink, recent, in_place, weights=w.copy())


def test_without_weights_or_kept(cuda_ok):
    """dst_weights and kept are optional; a second cut of what a cut left changes nothing."""
    dims, rows, _, w = setup("f16", 64, 32, 300, (300, 200), 2)
    d_rows, d_w = to_dev(rows), to_dev(w)
    lens = torch.tensor([300, 200], dtype=torch.int32, device=DEV)
    dst, dlen = torch.zeros(2, 50, 128, dtype=torch.uint8, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    q.qsvd_evict_rows(dims, d_w, lens, 50, d_rows, sink=2, recent=3, dst_max_len=50, dst_cache=dst, dst_lengths=dlen)
    q.qsvd_evict_rows(dims, d_w, lens, 50, d_rows, sink=2, recent=3)
    torch.cuda.synchronize()
    assert torch.equal(dst, d_rows[:, :50]) and dlen.tolist() == lens.tolist() == [50, 50]
    again = (d_rows.clone(), d_w.clone())
    q.qsvd_evict_rows(dims, d_w, lens, 50, d_rows, sink=2, recent=3)
    torch.cuda.synchronize()
    assert torch.equal(d_rows, again[0]) and torch.equal(d_w, again[1])


def test_graph_replay(cuda_ok):
    """A captured cut out of place, replayed on new weights."""
    dims, rows, _, w = setup("f16", 128, 32, 500, (500, 90, 333), 3)
    d_rows, d_w = to_dev(rows), to_dev(w)
    lens = torch.tensor([500, 90, 333], dtype=torch.int32, device=DEV)
    dst, dlen = torch.zeros(3, 100, 256, dtype=torch.uint8, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    kept = torch.zeros(3, 100, dtype=torch.int32, device=DEV)
    ws = torch.empty(q.evict_workspace_bytes(dims, 100), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        q.qsvd_evict_rows(dims, d_w, lens, 100, d_rows, sink=1, recent=20, dst_max_len=100, dst_cache=dst, dst_lengths=dlen,
                          kept=kept, workspace=ws)
    for seed in (4, 5):
        w2 = setup("f16", 128, 32, 500, (500, 90, 333), seed)[3]
        d_w.copy_(torch.from_numpy(w2))
        graph.replay()
        torch.cuda.synchronize()
        for b, n in enumerate((500, 90, 333)):
            at = keep_rows(w2[b, :n], n, 100, 1, 20)
            assert kept[b, :len(at)].tolist() == at
            assert np.array_equal(dst[b, :len(at)].cpu().numpy(), rows[b, at])


@pytest.mark.parametrize("in_place", [True, False])
def test_caches_beyond_32_bit_offsets(cuda_ok, in_place):
    """Two sequences of 800,000 rows of 3 KB: bytes past 2^32, rows compared with a gather by the kept indices."""
    B, n, r, budget = 2, 800_000, 1536, 700_000
    dims = q.make_dims(64, 1, 64, r, B, n, cache="f16")
    rows = torch.arange(B * n, device=DEV, dtype=torch.int64)
    cache = ((rows[:, None] * 7 + torch.arange(r, device=DEV)) % 2039).to(torch.float16).view(B, n, r)
    w = torch.rand(B, n, device=DEV)
    w0 = w.clone()
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    kept = torch.zeros(B, budget, dtype=torch.int32, device=DEV)
    if in_place:
        q.qsvd_evict_rows(dims, w, lens, budget, cache, sink=4, recent=1000, kept=kept)
        got = cache
    else:
        got = torch.zeros(B, budget, r, dtype=torch.float16, device=DEV)
        q.qsvd_evict_rows(dims, w, lens, budget, cache, sink=4, recent=1000, kept=kept, dst_max_len=budget, dst_cache=got,
                          dst_lengths=torch.zeros_like(lens))
    torch.cuda.synchronize()
    for b in range(B):
        key = w0[b].clone()
        key[:4] = key[n - 1000:] = 2.0
        want = torch.sort(key, descending=True, stable=True).indices[:budget].sort().values
        assert torch.equal(kept[b].long(), want)
        values = ((want[:, None] + b * n) * 7 + torch.arange(r, device=DEV)) % 2039
        assert torch.equal(got[b, :budget], values.to(torch.float16))
        del values


def test_two_cuts_at_once(cuda_ok):
    """Two batches cut in place on two streams."""
    sets = []
    for seed in (1, 2):
        dims, rows, _, w = setup("f16", 256, 128, 3000, (3000, 2500, 100), seed)
        sets.append((dims, rows, w, to_dev(rows), to_dev(w), torch.tensor([3000, 2500, 100], dtype=torch.int32, device=DEV),
                     torch.empty(q.evict_workspace_bytes(dims, 900), dtype=torch.uint8, device=DEV), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for dims, _, _, d_rows, d_w, lens, ws, st in sets:
        q.qsvd_evict_rows(dims, d_w, lens, 900, d_rows, sink=3, recent=64, workspace=ws, stream=st)
    torch.cuda.synchronize()
    for _, rows, w, d_rows, _, lens, _, _ in sets:
        assert lens.tolist() == [900, 900, 100]
        for b, n in enumerate((3000, 2500, 100)):
            at = keep_rows(w[b, :n], n, 900, 3, 64)
            assert np.array_equal(d_rows[b, :len(at)].cpu().numpy(), rows[b, at])
