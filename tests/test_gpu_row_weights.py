"""qsvd_decode_attn_weights: a decode step that also gives each row's attention
weight.  The output is the plain decode's within the decode's bar; the
weights are compared with the definition in 64 bits, within a bound on the
scores' error that is computed from the inputs."""
import pytest
import torch

import rank_joint_qkv_b200 as q
from tests.serving_util import DEV, Layer, close_weights, rel_err

pytestmark = pytest.mark.gpu

A, S, T, C = (q.QSVD_KERNEL_AUTO, q.QSVD_KERNEL_SIMT, q.QSVD_KERNEL_TCGEN05_CTA, q.QSVD_KERNEL_TCGEN05_CLUSTER)
CASES = {
    # every split kernel; head padding (H 4 of 16, 20 of 32), lengths 0, 1, either side of a tile
    "f32-simt": dict(cache="f32", weight="f32", H=4, d_h=64, r=96, lens=(5, 0, 1, 130)),
    "f16-simt": dict(cache="f16", H=6, d_h=64, r=160, lens=(127, 128, 129), kernel=S),
    "f16-tc": dict(cache="f16", H=4, d_h=64, r=256, lens=(0, 1, 127, 128, 129, 700), kernel=T),
    "f16-tc-20-heads": dict(cache="f16", H=20, d_h=64, r=384, lens=(300, 64), kernel=T),
    "bf16-tc": dict(cache="bf16", weight="bf16", out="bf16", H=32, d_h=128, r=512, lens=(1000, 3), kernel=T),
    # three parts of the absorbed query: both head paddings, all of TMEM, both absorption kernels, two parts by cluster
    "bf16-7b": dict(cache="bf16", weight="bf16", out="bf16", H=32, d_h=128, r=1536, lens=(300, 0, 128, 1), kernel=T),
    "bf16-12-heads": dict(cache="bf16", weight="f16", H=12, d_h=64, r=640, lens=(129, 20), kernel=T),
    "bf16-f32-weights": dict(cache="bf16", weight="f32", H=4, d_h=64, r=128, lens=(0, 140), kernel=T),
    "bf16-d-24": dict(cache="bf16", weight="bf16", H=8, d_h=24, r=256, lens=(130, 3), kernel=T),
    "bf16-cluster": dict(cache="bf16", weight="bf16", H=8, d_h=64, r=512, lens=(0, 257, 40), kernel=C),
    "f16-cluster": dict(cache="f16", H=8, d_h=64, r=512, lens=(0, 257, 40), kernel=C),
    "i8-tc": dict(cache="i8", H=4, d_h=64, r=256, lens=(0, 1, 129, 500), kernel=T),
    "i8-tc-32-heads": dict(cache="i8", weight="bf16", out="bf16", H=32, d_h=64, r=256, lens=(200, 77), kernel=T),
    "i4-tc": dict(cache="i4", H=8, d_h=64, r=384, lens=(1, 400), kernel=T),
    "i4-simt-group": dict(cache="i4", H=4, d_h=64, r=96, group=32, lens=(33, 9), kernel=S),
    "f16-rope-tc": dict(cache="f16", H=4, d_h=128, r=256, lens=(0, 1, 129, 333), rope=True),
    "bf16-rope-tc": dict(cache="bf16", weight="bf16", out="bf16", H=8, d_h=128, r=128, lens=(130, 64), rope=True),
    "f32-rope-simt": dict(cache="f32", weight="f32", H=2, d_h=64, r=64, lens=(40, 0, 17), rope=True),
}


@pytest.mark.parametrize("name", list(CASES))
def test_weights_against_the_definition(cuda_ok, name):
    m = Layer(**CASES[name])
    plain = m.empty_out()
    q.qsvd_decode_attn(m.dims, m.packed, m.qin, True, m.cache, m.scales, m.lengths, plain)
    _, want, bound = m.exact()
    w = torch.full((m.B, m.max_len), 7.0, device=DEV)   # written, not added to
    out = m.empty_out()
    ws = q.qsvd_decode_attn_weights(m.dims, m.packed, m.qin, True, m.cache, m.scales, m.lengths, out, w,
                                    accumulate=False)
    torch.cuda.synchronize()
    if not (torch.isfinite(out).all() and rel_err(out, plain) <= 2e-3 + torch.finfo(out.dtype).eps * 8):
        raise AssertionError(rel_err(out, plain))   # 16-bit outputs: one step of an output 8 rms large
    assert q.status_word(ws) == 0
    close_weights(w, want, bound, m.lens)
    for b, n in enumerate(m.lens):
        assert bool((w[b, n:] == 7.0).all())            # entries behind the length stay
    # added to what is there: one float32 addition of the same sum
    before = torch.rand(m.B, m.max_len, device=DEV)
    acc = before.clone()
    q.qsvd_decode_attn_weights(m.dims, m.packed, m.qin, True, m.cache, m.scales, m.lengths, out, acc, workspace=ws)
    torch.cuda.synchronize()
    for b, n in enumerate(m.lens):
        assert torch.equal(acc[b, :n], before[b, :n] + w[b, :n])
        assert torch.equal(acc[b, n:], before[b, n:])


@pytest.mark.parametrize("kernel", [S, T])
def test_rows_behind_the_length_have_no_bearing(cuda_ok, kernel):
    """NaN and infinity behind each length; the weights of a sequence sum to H."""
    clean = Layer(H=4, r=256, lens=(100, 1, 260), kernel=kernel, seed=3)
    for past in (float("nan"), float("inf")):
        m = Layer(H=4, r=256, lens=(100, 1, 260), kernel=kernel, seed=3, past=past)
        got = []
        for layer in (clean, m):
            w, out = torch.zeros(3, layer.max_len, device=DEV), layer.empty_out()
            q.qsvd_decode_attn_weights(layer.dims, layer.packed, layer.qin, True, layer.cache, None, layer.lengths, out, w)
            got.append((out, w))
        torch.cuda.synchronize()
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
        # H probabilities' sums, each 1 up to the rounding of n float32 terms
        assert bool(((got[1][1].double().sum(1) - 4).abs() <= 4 * 300 * 2.0 ** -23).all())


def test_split_counts_give_the_same_weights(cuda_ok):
    m = Layer(H=4, r=256, lens=(700, 129), kernel=T)
    _, want, bound = m.exact()
    for splits in (1, 3, 1000):
        w, out = torch.zeros(2, m.max_len, device=DEV), m.empty_out()
        q.qsvd_decode_attn_weights(m.dims, m.packed, m.qin, True, m.cache, None, m.lengths, out, w, num_splits=splits)
        close_weights(w, want, bound, m.lens)


def test_graph_replay_and_side_stream(cuda_ok):
    """Captured on a side stream and replayed: each replay adds the same weights; two graphs with workspaces of their own."""
    m = Layer(H=8, r=256, lens=(300, 40), kernel=T)
    once, out = torch.zeros(2, m.max_len, device=DEV), m.empty_out()
    q.qsvd_decode_attn_weights(m.dims, m.packed, m.qin, True, m.cache, None, m.lengths, out, once)
    accs, graphs = [], []
    side = torch.cuda.Stream()
    for _ in range(2):
        acc, o = torch.zeros(2, m.max_len, device=DEV), m.empty_out()
        ws = torch.empty(q.decode_weights_workspace_bytes(m.dims), dtype=torch.uint8, device=DEV)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            q.qsvd_decode_attn_weights(m.dims, m.packed, m.qin, True, m.cache, None, m.lengths, o, acc, workspace=ws)
        accs.append((acc, o, ws))
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    want = (once + once) + once
    for acc, o, _ in accs:
        assert torch.equal(acc, want) and torch.equal(o, out)


def test_clamped_length_is_flagged(cuda_ok):
    m = Layer(H=4, r=256, lens=(50, 60), kernel=T)
    lengths = torch.tensor([-3, m.max_len + 9], dtype=torch.int32, device=DEV)
    w, out = torch.zeros(2, m.max_len, device=DEV), m.empty_out()
    ws = q.qsvd_decode_attn_weights(m.dims, m.packed, m.qin, True, m.cache, None, lengths, out, w)
    assert q.status_word(ws) == q.QSVD_STATUS_LEN_CLAMPED
    assert bool((out[0] == 0).all()) and bool((w[0] == 0).all()) and bool((w[1] > 0).all())


@pytest.mark.parametrize("prefix", [0, 1])
def test_bf16_rows_see_more_of_the_query_than_two_parts(cuda_ok, prefix):
    """Rows V c_j - U c_k whose two large terms nearly cancel, for queries with 24 significant bits.  With u = 2^-23 a term's
    product of query and weight comes from three parts (three truncations) and one scaling (u / 2), and enters the score's
    sum with one more truncation: 4.5 u of each term.  The gain on the query moves a score by less than 2^-19 of itself;
    2^-20 for the exponential, the sums and the float32 weights.  Two parts would miss up to 2^-18 of each term."""
    B, n, r, d_h = 8, 64, 256, 64
    g = torch.Generator()
    g.manual_seed(3)
    bf = lambda x: x.bfloat16().double()  # noqa: E731
    a = bf(1 + torch.rand(r, generator=g))
    rows = torch.zeros(n, r, dtype=torch.float64)
    pairs = []
    for t in range(1, n):   # U is what bf16 has next to V a_j / a_k
        j, k = 2 * t, 2 * t + 1
        for _ in range(1000):
            v = float(bf(256 + 256 * torch.rand(1, generator=g)))
            u = float(bf(torch.tensor(v * float(a[j] / a[k]))))
            if abs(v * a[j] - u * a[k]) < 4:
                break
        rows[t, j], rows[t, k] = v, -u
        pairs.append((j, k))
    query = (1 + torch.rand(B, generator=g)).float()
    dims = q.make_dims(d_h, 1, d_h, r, B, n, cache="bf16", weight="bf16", kernel=T)
    wuk = torch.zeros(r, d_h, dtype=torch.float64)
    wuk[:, 0] = a
    z = torch.zeros(r, d_h, device=DEV, dtype=torch.bfloat16)
    packed = q.qsvd_prepare_weights(dims, z.t().contiguous(), z, wuk.bfloat16().to(DEV), z)
    qin = torch.zeros(B, d_h)
    qin[:, 0] = query
    cache = rows.bfloat16()[None].repeat(B, 1, 1).contiguous().to(DEV)
    lengths = torch.full((B,), n, dtype=torch.int32, device=DEV)
    w, out = torch.zeros(B, n, device=DEV), torch.zeros(B, d_h, device=DEV)
    zero = torch.zeros(1, r, device=DEV, dtype=torch.bfloat16)
    q.qsvd_decode_attn_shared(dims, packed, qin.to(DEV), False, zero if prefix else None, None, prefix, cache, None, lengths,
                              out, weights=w, accumulate=False)
    scores = query.double()[:, None] * (rows @ a)[None] / d_h ** 0.5
    terms = query.double()[:, None] * (rows.abs() @ a)[None] / d_h ** 0.5
    lim = 4.5 * 2.0 ** -23 * terms + 2.0 ** -19 * scores.abs() + 2.0 ** -20
    got = w.double().cpu()
    off = (got[:, 1:] / got[:, :1]).log() - scores[:, 1:]
    assert float((off.abs() / lim[:, 1:]).max()) <= 1.0
    # by arithmetic: with two parts of the absorbed query some of these rows would be further off than that
    qt = query.double()[:, None] * a[None] * (1.4426950408889634 / d_h ** 0.5)
    two = bf(qt) + bf(qt - bf(qt))
    miss = ((two - qt) @ rows.t()) * 0.6931471805599453
    assert float((miss[:, 1:].abs() / lim[:, 1:]).max()) > 1.5


@pytest.mark.parametrize("kernel,H,r", [(T, 1, 256), (C, 1, 256), (C, 12, 512), (C, 20, 1024), (A, 32, 1792), (A, 32, 2048)])
@pytest.mark.parametrize("n", [64, 700])
def test_bf16_rows_see_more_of_the_query_on_every_kernel(cuda_ok, kernel, H, r, n):
    """The rows of the test above, their two terms in any two channels and the heads alike, on the one-CTA kernel, on
    clusters of two to eight CTAs, and where the latter is the library's own choice.  The same bounds, and H additions of the
    heads' equal weights in each of the two weights compared."""
    B, d_h = 4, 64
    g = torch.Generator()
    g.manual_seed(7)
    bf = lambda x: x.bfloat16().double()  # noqa: E731
    a = bf(1 + torch.rand(r, generator=g))
    rows = torch.zeros(n, r, dtype=torch.float64)
    for t in range(1, n):
        for _ in range(1000):
            j, k = torch.randperm(r, generator=g)[:2].tolist()
            v = float(bf(256 + 256 * torch.rand(1, generator=g)))
            u = float(bf(torch.tensor(v * float(a[j] / a[k]))))
            if abs(v * a[j] - u * a[k]) < 4:
                break
        rows[t, j], rows[t, k] = v, -u
    query = (1 + torch.rand(B, generator=g)).float()
    E = H * d_h
    dims = q.make_dims(E, H, d_h, r, B, n, cache="bf16", weight="bf16", kernel=kernel)
    wuk = torch.zeros(r, E, dtype=torch.float64)
    wuk[:, ::d_h] = a[:, None]
    z = torch.zeros(r, E, device=DEV, dtype=torch.bfloat16)
    packed = q.qsvd_prepare_weights(dims, z.t().contiguous(), z, wuk.bfloat16().to(DEV), z)
    qin = torch.zeros(B, E)
    qin[:, ::d_h] = query[:, None]
    cache = rows.bfloat16()[None].repeat(B, 1, 1).contiguous().to(DEV)
    lengths = torch.full((B,), n, dtype=torch.int32, device=DEV)
    w, out = torch.zeros(B, n, device=DEV), torch.zeros(B, E, device=DEV)
    ws = q.qsvd_decode_attn_weights(dims, packed, qin.to(DEV), False, cache, None, lengths, out, w, accumulate=False)
    torch.cuda.synchronize()
    status, _, _, ran = ws[:16].view(torch.int32).tolist()
    assert status == 0 and ran == (T if kernel == T else C)
    scores = query.double()[:, None] * (rows @ a)[None] / d_h ** 0.5
    terms = query.double()[:, None] * (rows.abs() @ a)[None] / d_h ** 0.5
    lim = 4.5 * 2.0 ** -23 * terms + 2.0 ** -19 * scores.abs() + 2.0 ** -20 + 2 * H * 2.0 ** -24
    got = w.double().cpu()
    off = (got[:, 1:] / got[:, :1]).log() - scores[:, 1:]
    assert float((off.abs() / lim[:, 1:]).max()) <= 1.0
    qt = query.double()[:, None] * a[None] * (1.4426950408889634 / d_h ** 0.5)
    two = bf(qt) + bf(qt - bf(qt))
    miss = ((two - qt) @ rows.t()) * 0.6931471805599453
    assert float((miss[:, 1:].abs() / lim[:, 1:]).max()) > 1.5


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("form", [dict(H=32, r=2048), dict(H=20, r=1792), dict(H=12, r=1024), dict(H=32, r=512)],
                         ids=["8-ctas-one-buffer", "7-ctas-one-buffer", "4-ctas", "2-ctas-one-buffer"])
def test_clusters_that_walk_many_tiles(cuda_ok, form, splits):
    """The exchange buffers of the cluster kernel used over and over, one of them or two, from one cluster to all that fit."""
    m = Layer(cache="bf16", weight="bf16", d_h=64, lens=(2500, 0, 1300, 128), kernel=C, seed=8, **form)
    want, want_w, bound = m.exact()
    w, out = torch.zeros(m.B, m.max_len, device=DEV), m.empty_out()
    ws = q.qsvd_decode_attn_weights(m.dims, m.packed, m.qin, True, m.cache, None, m.lengths, out, w, accumulate=False,
                                    num_splits=splits)
    torch.cuda.synchronize()
    assert q.status_word(ws) == 0
    assert rel_err(out, want) <= 2e-3
    close_weights(w, want_w, bound, m.lens)
    plain = m.empty_out()
    q.qsvd_decode_attn(m.dims, m.packed, m.qin, True, m.cache, None, m.lengths, plain, num_splits=splits)
    assert rel_err(out, plain) <= 2e-3
