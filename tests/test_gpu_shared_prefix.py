"""qsvd_decode_attn_shared: a batch over a shared prefix and its own rows, against
the definition in 64 bits, and the three serving calls used together."""
import numpy as np
import pytest
import torch

import rank_joint_qkv_b200 as q
from tests.serving_util import DEV, TORCH, Layer, close_weights, keep_rows, rel_err

pytestmark = pytest.mark.gpu

S = q.QSVD_KERNEL_SIMT
CASES = {
    # the prefix's tiles (256 tokens) and K blocks (64) met exactly, missed by one, and of one row; idle query rows
    "f16-1": dict(prefix=1, lens=(5, 0, 130)),
    "f16-63": dict(prefix=63, lens=(0, 0, 0)),
    "f16-64": dict(prefix=64, lens=(1,)),
    "f16-65": dict(prefix=65, lens=(128, 129), H=8),
    "f16-255": dict(prefix=255, lens=(3, 4, 5, 6, 7), H=32),
    "f16-256": dict(prefix=256, lens=(64,) * 33, H=4),                  # 33 sequences, 32 to a block
    "f16-257": dict(prefix=257, lens=(9, 700), H=20, r=384),            # 6 sequences to a block, 120 of 128 rows
    "f16-1500": dict(prefix=1500, lens=(40, 0, 300, 1, 2), H=32, d_h=128, r=1536),
    "f16-5000": dict(prefix=5000, lens=(10,) * 9, H=16, r=512),
    "f16-no-prefix": dict(prefix=0, lens=(5, 0, 130)),
    "f16-64-heads": dict(prefix=700, lens=(30, 2), H=64, r=128),        # own rows on the CUDA cores
    "f16-128-heads": dict(prefix=300, lens=(10, 0), H=128, r=64),
    "f16-rank-192": dict(prefix=520, lens=(65, 1), H=6, r=192),         # a ragged block of 256 channels
    "bf16": dict(cache="bf16", weight="bf16", out="bf16", prefix=900, lens=(0, 33, 200), H=32, r=512),
    "bf16-f32-out": dict(cache="bf16", weight="bf16", prefix=300, lens=(20, 1)),
    "i8": dict(cache="i8", prefix=777, lens=(0, 130, 5), H=8, r=256),
    "i8-bf16": dict(cache="i8", weight="bf16", out="bf16", prefix=1029, lens=(64, 64), H=32, r=768),
    "i4": dict(cache="i4", prefix=500, lens=(1, 129), r=384),
    "i4-group": dict(cache="i4", prefix=130, lens=(40, 3), r=192, group=64),
    "mixed-weights": dict(cache="f16", weight="f32", prefix=400, lens=(20, 60)),
    "f16-cluster": dict(prefix=300, lens=(0, 257, 40), H=8, r=512, kernel=q.QSVD_KERNEL_TCGEN05_CLUSTER),
    "f16-pairs": dict(prefix=9300, lens=(3, 0, 130) * 6, H=32, r=128),   # 5 blocks of query rows in pairs, 37 tiles
    "bf16-pairs": dict(cache="bf16", weight="bf16", out="bf16", prefix=10001, lens=(1,) * 16, H=32, r=192),
    "i8-pairs": dict(cache="i8", prefix=9999, lens=(20,) * 16, H=32, r=256),
    "f16-rank-4096": dict(prefix=130, lens=(3, 0, 40), H=4, r=4096),    # eight k-splits of the projections: one cluster
    "f16-rank-4160": dict(prefix=130, lens=(3, 0) * 9, H=4, r=4160),    # nine: tickets; two blocks of sequences
    "bf16-rank-4160": dict(cache="bf16", weight="bf16", prefix=70, lens=(3, 20), H=4, r=4160),
    # CUDA cores: fp32 rows, other ranks, by request, more heads than a block has rows
    "f32": dict(cache="f32", weight="f32", prefix=300, lens=(0, 140, 7), r=96),
    "f16-simt": dict(prefix=300, lens=(5, 0), kernel=S),
    "f16-rank-96": dict(prefix=129, lens=(5, 0), r=96),
    "i8-simt": dict(cache="i8", prefix=129, lens=(70, 2), r=96, group=32, kernel=S),
    "f16-130-heads": dict(prefix=70, lens=(5, 9), H=130, d_h=64, r=64),
    # rotary: positions run through the prefix and on into the own rows, past the packed table's end
    "rope-1": dict(prefix=1, lens=(5, 0, 130), d_h=128, rope=True),
    "rope-127": dict(prefix=127, lens=(0, 0, 0), d_h=128, rope=True),
    "rope-129": dict(prefix=129, lens=(1,), H=3, d_h=128, r=64, rope=True),      # an odd head: half a pair
    "rope-256": dict(prefix=256, lens=(64,) * 33, H=4, d_h=128, r=128, rope=True),
    "rope-1500": dict(prefix=1500, lens=(40, 0, 300, 1, 2), H=32, d_h=128, r=1536, rope=True),
    "rope-no-prefix": dict(prefix=0, lens=(5, 0, 130), d_h=128, rope=True),
    "rope-bf16": dict(cache="bf16", weight="bf16", out="bf16", prefix=2000, lens=(0, 33, 200), H=20, d_h=128, r=512, rope=True),
    "rope-pairs": dict(prefix=9300, lens=(3, 0, 130) * 6, H=32, d_h=128, r=128, rope=True),
    "rope-130-heads": dict(prefix=70, lens=(5, 9), H=130, d_h=128, r=64, rope=True),   # the prefix on the CUDA cores
    "rope-f32": dict(cache="f32", weight="f32", prefix=140, lens=(0, 30, 7), H=2, r=96, rope=True),
    "rope-i8": dict(cache="i8", prefix=129, lens=(70, 2), H=2, d_h=128, r=128, rope=True),
    "rope-d-64": dict(prefix=150, lens=(5, 0), rope=True),
    "rope-simt": dict(prefix=130, lens=(5, 0), H=2, d_h=128, r=128, rope=True, kernel=S),
    # the combine without the tensor-core GEMV (d_h % 64 != 0)
    "f16-d-24": dict(prefix=300, lens=(5, 0, 40), H=8, d_h=24, r=128),
    "f32-d-24": dict(cache="f32", weight="f32", prefix=3, lens=(0, 2), H=8, d_h=24, r=64),
}


def run(m, weights=None, accumulate=False, splits=0):
    out = m.empty_out()
    ws = q.qsvd_decode_attn_shared(m.dims, m.packed, m.qin, True, m.prefix, m.prefix_scales, m.prefix_values.shape[0],
                                   m.cache, m.scales, m.lengths, out, weights=weights, accumulate=accumulate,
                                   num_splits=splits)
    torch.cuda.synchronize()
    assert q.status_word(ws) == 0
    return out


def close_out(m, out, want):
    """The decode's bar, 2e-3 of rms (1e-4 for fp32 rows), half a step of a
    16-bit output, and the rounding of P: with p_t entering the value product
    as p_t (1 + d_t), |d_t| <= u, and the softmax's sum unrounded, an output
    moves by sum_t p_t d_t v_t, at most u sum_t p_t |v_t|.  u is half a step of
    fp16, 2^-11, for fp16 rows (one row that takes all the weight shows it
    whole, whatever the output's rms); twice that for quantised ones, whose
    own rows are rounded to fp16 too; 2^-16 for bf16's two parts."""
    assert torch.isfinite(out).all()
    dt = m.cache.dtype
    bar = 1e-4 if dt == torch.float32 else 2e-3
    u = {torch.float32: 0.0, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -16}.get(dt, 2.0 ** -10)
    half = torch.finfo(out.dtype).eps / 2 if out.dtype != torch.float32 else 0.0
    rms = float(want.square().mean().sqrt())
    lim = bar * rms + half * want.abs() + u * m.spread + 1e-30
    worst = float(((out.double() - want).abs() / lim).max())
    assert worst <= 1.0, worst


@pytest.mark.parametrize("name", list(CASES))
def test_against_the_definition(cuda_ok, name):
    m = Layer(**CASES[name])
    want, want_w, bound = m.exact()
    w = torch.full((m.B, m.max_len), 7.0, device=DEV)
    out = run(m, weights=w)
    close_out(m, out, want)
    # twice the accumulations per prefix score: hi and lo parts go into one accumulator
    close_weights(w, want_w, 3 * bound, m.lens)
    for b, n in enumerate(m.lens):
        assert bool((w[b, n:] == 7.0).all())
    # weights are optional; without them bf16 weights take the query in two parts instead of three (2^-16 of it)
    again = run(m)
    assert torch.equal(again, out) if m.weight != "bf16" else rel_err(again, out) <= 2e-3 + 8 * torch.finfo(out.dtype).eps


@pytest.mark.parametrize("cache", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("rise", [1.0, -1.0])
def test_tile_references_that_differ(cuda_ok, cache, rise):
    """Rows growing (or shrinking) along the prefix, so that tiles' maxima lie tens of log2 units apart."""
    m = Layer(cache=cache, weight="bf16" if cache == "bf16" else "f16", prefix=2100, lens=(30, 0, 5), H=8, r=256, peak=1.0)
    ramp = torch.linspace(0.2, 12.0, 2100, device=DEV)[:, None]
    ramp = ramp if rise > 0 else ramp.flip(0)
    if cache == "i8":
        m.prefix_scales = (m.prefix_scales.float() * ramp).half()
        m.prefix_values = (m.prefix.double().view(2100, -1, 128) * m.prefix_scales.double()[..., None]).view(2100, -1)
    else:
        m.prefix = (m.prefix.float() * ramp).to(TORCH[cache])
        m.prefix_values = m.prefix.double()
    want, want_w, bound = m.exact()
    w = torch.zeros(m.B, m.max_len, device=DEV)
    out = run(m, weights=w)
    close_out(m, out, want)
    close_weights(w, want_w, 3 * bound, m.lens)


@pytest.mark.parametrize("cache", ["f16", "bf16"])
def test_rotary_rows_of_very_different_size(cuda_ok, cache):
    """Zero rows, rows 2^-12 and 8 times the usual (scores up to eight times the peak), a zero query, one 64 times the usual
    (one row takes all the weight)."""
    m = Layer(cache=cache, weight=cache, prefix=700, lens=(30, 0, 5), H=4, d_h=128, r=256, peak=0.5, rope=True)
    size = torch.tensor([0.0, 2.0 ** -12, 1.0, 8.0], device=DEV).repeat(175)[:, None]
    m.prefix = (m.prefix.float() * size).to(TORCH[cache])
    m.prefix_values = m.prefix.double()
    m.qin[0] = 0
    m.qin[2] *= 64
    want, want_w, bound = m.exact()
    w = torch.zeros(m.B, m.max_len, device=DEV)
    out = run(m, weights=w)
    close_out(m, out, want)
    close_weights(w, want_w, 3 * bound, m.lens)


FORMS = [dict(H=8, r=256), dict(H=4, d_h=128, r=256, rope=True)]


@pytest.mark.parametrize("form", FORMS, ids=["absorbed", "rope"])
def test_same_as_a_decode_over_the_whole_rows(cuda_ok, form):
    """The prefix copied in front of every sequence's rows gives the plain decode's output."""
    m = Layer(prefix=600, lens=(40, 0, 333), **form)
    whole = Layer(lens=[600 + n for n in m.lens], **form)
    for b, n in enumerate(m.lens):
        whole.cache[b, :600] = m.prefix
        whole.cache[b, 600:600 + n] = m.cache[b, :n]
    plain = whole.empty_out()
    packed = q.qsvd_prepare_weights(whole.dims, m.wd, m.wuq, m.wuk, m.wuv)
    q.qsvd_decode_attn(whole.dims, packed, m.qin, True, whole.cache, None, whole.lengths, plain)
    assert rel_err(run(m), plain) <= 2e-3


@pytest.mark.parametrize("proj", ["chain", "fold"])
def test_output_projection(cuda_ok, proj):
    m = Layer(prefix=300, lens=(20, 0, 5), H=4, r=128, out_proj=proj)
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    wo = (torch.randn(m.E, m.E, generator=g, device=DEV) / m.E ** 0.5).half()
    q.qsvd_prepare_out_proj(m.dims, wo, m.packed)
    want, _, _ = m.exact(wo)
    # the fold's stored factors are rounded once (2^-11 each): their share of the output, doubled for the bar's max
    extra = 0.0 if proj == "chain" else 2.0 ** -10
    assert rel_err(run(m), want) <= 2e-3 + extra


def test_rows_behind_the_length_have_no_bearing(cuda_ok):
    for form in (dict(), dict(kernel=S), dict(d_h=128, rope=True)):
        clean = run(Layer(prefix=100, lens=(10, 0, 129), **form))
        dirty = run(Layer(prefix=100, lens=(10, 0, 129), past=float("nan"), **form))
        assert torch.equal(clean, dirty)


def test_a_strided_view_of_a_longer_prefix(cuda_ok):
    """The prefix may lie inside a larger buffer: rows behind prefix_len are not read."""
    m = Layer(prefix=300, lens=(10, 20))
    out = run(m)
    room = torch.full((400, m.r), float("nan"), device=DEV, dtype=torch.float16)
    room[50:350] = m.prefix
    m.prefix = room[50:350]
    assert torch.equal(run(m), out)


@pytest.mark.parametrize("form", FORMS, ids=["absorbed", "rope"])
def test_graph_replay_on_a_side_stream(cuda_ok, form):
    """Two graphs with workspaces of their own, replayed in turn with new queries and lengths."""
    m = Layer(prefix=700, lens=(40, 3, 200), **form)
    side, graphs = torch.cuda.Stream(), []
    for _ in range(2):
        out, w = m.empty_out(), torch.zeros(m.B, m.max_len, device=DEV)
        ws = torch.empty(q.decode_shared_workspace_bytes(m.dims, 700), dtype=torch.uint8, device=DEV)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            q.qsvd_decode_attn_shared(m.dims, m.packed, m.qin, True, m.prefix, None, 700, m.cache, None, m.lengths, out,
                                      weights=w, accumulate=False, workspace=ws)
        graphs.append((graph, out, w, ws))
    for lens in ((40, 3, 200), (0, 207, 1)):
        m.qin.mul_(0.9)
        m.lens = list(lens)
        m.lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        for graph, *_ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want, want_w, bound = m.exact()
        for _, out, w, _ in graphs:
            close_out(m, out, want)
            close_weights(w, want_w, 3 * bound, m.lens)


@pytest.mark.parametrize("cache", ["f16", "i8"])
def test_decode_cut_append_decode(cuda_ok, cache):
    """As they are used: steps that add up weights over a shared prefix, a cut of the own rows, a new token appended
    behind the kept rows, and a step over what is left."""
    budget, sink, recent = 48, 2, 8
    m = Layer(cache=cache, prefix=500, lens=(120, 48, 90), H=8, r=256, room=30)
    acc = torch.zeros(m.B, m.max_len, device=DEV)
    want_acc = torch.zeros(m.B, m.max_len, device=DEV, dtype=torch.float64)
    bounds = []
    for step in range(3):
        m.qin = m.qin.roll(1, 0).contiguous()
        run(m, weights=acc, accumulate=True)
        _, w, bound = m.exact()
        want_acc += w
        bounds.append(bound)
    close_weights(acc, want_acc, 3 * max(bounds), m.lens)
    kept = torch.zeros(m.B, budget, dtype=torch.int32, device=DEV)
    before = acc.cpu().numpy()
    q.qsvd_evict_rows(m.dims, acc, m.lengths, budget, m.cache, m.scales, sink=sink, recent=recent, kept=kept)
    torch.cuda.synchronize()
    rows = [keep_rows(before[b, :n], n, budget, sink, recent) for b, n in enumerate(m.lens)]
    for b, at in enumerate(rows):
        assert kept[b, :len(at)].tolist() == at
        m.values[b, :len(at)] = m.values[b, at].clone()
    assert m.lengths.tolist() == [len(at) for at in rows]
    # the next token's row goes behind the kept ones
    x = torch.randn(m.B, m.E, device=DEV).to(m.wd.dtype)
    c = torch.zeros(m.B, m.r, device=DEV)
    q.qsvd_append_latent(m.dims, m.packed, x, m.lengths, m.cache, m.scales, c)
    m.lengths += 1
    torch.cuda.synchronize()
    for b, at in enumerate(rows):
        row = m.cache[b, len(at)].double()
        if cache == "i8":
            row = (row.view(-1, 128) * m.scales[b, len(at)].double()[:, None]).view(-1)
        m.values[b, len(at)] = row
    m.lens = [len(at) + 1 for at in rows]
    w = acc.clone()
    out = run(m, weights=w, accumulate=True)
    want, want_w, bound = m.exact()
    close_out(m, out, want)
    for b, n in enumerate(m.lens):
        assert bool((w[b, n:] == 0).all())   # the cut left zeros for the rows to come
    # a float32 sum of two terms: the new weights come back up to one rounding of the sum
    close_weights(w - acc, want_w, 3 * bound + 2.0 ** -23 * float(w.max()) / max(float(want_w[want_w > 0].min()), 1e-30), m.lens)


def test_empty_everything_gives_zero_rows(cuda_ok):
    m = Layer(prefix=0, lens=(0, 0))
    assert bool((run(m) == 0).all())
    m = Layer(prefix=0, lens=(0, 3), H=8, d_h=24, r=64)
    assert bool((run(m)[0] == 0).all())


@pytest.mark.parametrize("form", FORMS, ids=["absorbed", "rope"])
def test_two_calls_at_once(cuda_ok, form):
    """Two batches on two streams with workspaces of their own, over one prefix, many times over."""
    a, b = (Layer(prefix=1200, lens=lens, max_len=1000, seed=5, **form) for lens in ((300, 0, 77), (10, 900, 128)))
    b.prefix, b.prefix_values, b.packed = a.prefix, a.prefix_values, a.packed
    b.wuq, b.wuk, b.wuv = a.wuq, a.wuk, a.wuv
    want = [run(m) for m in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[m.empty_out() for _ in range(20)] for m in (a, b)]
    wss = [torch.empty(q.decode_shared_workspace_bytes(m.dims, 1200), dtype=torch.uint8, device=DEV) for m in (a, b)]
    torch.cuda.synchronize()
    for i in range(20):
        for m, st, o, ws in zip((a, b), streams, outs, wss):
            q.qsvd_decode_attn_shared(m.dims, m.packed, m.qin, True, m.prefix, None, 1200, m.cache, None, m.lengths, o[i],
                                      workspace=ws, stream=st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for x in o:
            assert torch.equal(x, w)


@pytest.mark.parametrize("form", FORMS, ids=["absorbed", "rope"])
def test_one_workspace_for_prefixes_that_grow_and_shrink(cuda_ok, form):
    """Calls in a row without a wait between them, each laying its workspace out for its own prefix."""
    layers = [Layer(prefix=p, lens=(30, 0, 129), **form) for p in (900, 40, 0, 513)]
    outs = [m.empty_out() for m in layers]
    ws = torch.empty(max(q.decode_shared_workspace_bytes(m.dims, 900) for m in layers), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    for m, out in zip(layers, outs):
        q.qsvd_decode_attn_shared(m.dims, m.packed, m.qin, True, m.prefix, None, m.prefix_values.shape[0], m.cache, None,
                                  m.lengths, out, workspace=ws)
    torch.cuda.synchronize()
    for m, out in zip(layers, outs):
        close_out(m, out, m.exact()[0])


@pytest.mark.parametrize("form", [dict(H=8), dict(d_h=128, rope=True)], ids=["absorbed", "rope"])
def test_the_query_as_given(cuda_ok, form):
    """qin as the B x E query itself instead of the token's latent."""
    m = Layer(prefix=300, lens=(20, 0, 129), **form)
    query = m.qin.double() @ m.wuq.double()
    out = m.empty_out()
    q.qsvd_decode_attn_shared(m.dims, m.packed, query.float().contiguous(), False, m.prefix, None, 300, m.cache, None,
                              m.lengths, out)
    close_out(m, out, m.exact()[0])


def test_on_the_other_current_stream(cuda_ok):
    """The call goes to the stream that is current, ordered behind what that stream holds."""
    m = Layer(prefix=300, lens=(10, 20))
    want = run(m)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q0 = m.qin.clone()
    m.qin.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        m.qin.copy_(q0)
        out = m.empty_out()
        q.qsvd_decode_attn_shared(m.dims, m.packed, m.qin, True, m.prefix, None, 300, m.cache, None, m.lengths, out)
    side.synchronize()
    assert torch.equal(out, want)
    assert np.isfinite(out.float().cpu().numpy()).all()


@pytest.mark.parametrize("size", [2.0 ** 18, 2.0 ** -17], ids=["large", "small"])
@pytest.mark.parametrize("kernel", [q.QSVD_KERNEL_AUTO, S], ids=["tc", "simt"])
@pytest.mark.parametrize("cache", ["i8", "i4"])
def test_a_quantised_prefix_takes_a_query_of_any_size(cuda_ok, cache, kernel, size):
    """One prefix row c and one own row of zeros: the own row's weight is 1 / (1 + e^s), which gives the prefix's score s
    back.  The absorbed query qt is q a tau, past fp16's range or within its last subnormals, and c the other way round.
    With T = sum_j |qt_j c_j|: qt_j from three parts and a scaling is off by 4.5 x 2^-23, as two fp16 parts of a scaled row
    by another 2^-22; 3 x 16 accumulations of 16 products, each cut off below 2^-22 of T; 2^-19 of s for the gain.  The
    weight in float32, its exponentials and sum: 2^-20 of w, an error of s of 2^-20 / (1 - w)."""
    B, r, d_h, qmax = 8, 256, 64, 7
    g = torch.Generator()
    g.manual_seed(11)
    a = (1 + torch.rand(r, generator=g)).bfloat16().double() * size
    codes = torch.randint(-qmax, qmax + 1, (1, r), generator=g)
    tau = d_h ** -0.5
    # a scale that brings T to about 16, a multiple of fp16's smallest number
    sc = torch.tensor(16.0 / float((1.5 * tau * a.abs() * codes[0].abs()).sum()), dtype=torch.float64).half().clamp(min=2.0 ** -24)
    values = codes.double() * sc.double()
    assert float(values.abs().max()) < 65504
    query = (1 + torch.rand(B, generator=g)).float()
    dims = q.make_dims(d_h, 1, d_h, r, B, 1, cache=cache, weight="bf16", kernel=kernel)
    wuk, wuv = torch.zeros(r, d_h, dtype=torch.float64), torch.zeros(r, d_h, dtype=torch.float64)
    wuk[:, 0] = a
    wuv[:, 1] = torch.randn(r, generator=g, dtype=torch.float64).bfloat16().double()
    z = torch.zeros(r, d_h, device=DEV, dtype=torch.bfloat16)
    packed = q.qsvd_prepare_weights(dims, z.t().contiguous(), z, wuk.bfloat16().to(DEV), wuv.bfloat16().to(DEV))
    qin = torch.zeros(B, d_h)
    qin[:, 0] = query
    stored = codes if cache == "i8" else (codes[:, 0::2] & 0xF) | ((codes[:, 1::2] & 0xF) << 4)
    prefix = stored.to(torch.int8 if cache == "i8" else torch.uint8).contiguous().to(DEV)
    scales = sc.expand(1, r // 128).contiguous().to(DEV)
    own = torch.zeros(B, 1, prefix.shape[1], dtype=prefix.dtype, device=DEV)
    own_scales = torch.ones(B, 1, r // 128, dtype=torch.float16, device=DEV)
    w, out = torch.zeros(B, 1, device=DEV), torch.zeros(B, d_h, device=DEV)
    ws = q.qsvd_decode_attn_shared(dims, packed, qin.to(DEV), False, prefix, scales, 1, own, own_scales,
                                   torch.ones(B, dtype=torch.int32, device=DEV), out, weights=w, accumulate=False)
    torch.cuda.synchronize()
    assert q.status_word(ws) == 0
    qt = query.double()[:, None] * a[None] * tau
    s, terms = qt @ values[0], qt.abs() @ values[0].abs()
    assert 4 < float(terms.min()) and float(s.abs().max()) < 8   # neither score far from the own row's
    w = w[:, 0].double().cpu()
    p = torch.sigmoid(s)
    lim = (6.5 * 2.0 ** -23 + 48 * 2.0 ** -22) * terms + 2.0 ** -19 * s.abs() + 2.0 ** -20 / p
    assert float((((1 - w) / w).log() - s).abs().div(lim).max()) <= 1.0
    # the value: p within its score's error and one fp16 rounding, c W in two 16-bit parts of the merged latent
    want = p * (values[0] @ wuv[:, 1])
    bar = (lim + 2.0 ** -11) * want.abs() + 2.0 ** -14 * (p * (values[0].abs() @ wuv[:, 1].abs()))
    assert bool(((out[:, 1].double().cpu() - want).abs() <= bar).all())


@pytest.mark.parametrize("form", [dict(H=8, r=512, lens=(0, 257, 40)), dict(H=20, r=1024, lens=(130, 1)),
                                  dict(H=32, d_h=128, r=2048, lens=(3, 300), kernel=q.QSVD_KERNEL_AUTO)],
                         ids=["4-ctas", "4-ctas-20-heads", "auto"])
def test_bf16_own_rows_on_clusters(cuda_ok, form):
    """Own rows on the cluster kernel and the prefix's products, both from three parts of the query, and from two without weights."""
    m = Layer(**dict(dict(cache="bf16", weight="bf16", prefix=700, kernel=q.QSVD_KERNEL_TCGEN05_CLUSTER), **form))
    want, want_w, bound = m.exact()
    w = torch.zeros(m.B, m.max_len, device=DEV)
    close_out(m, run(m, weights=w), want)
    close_weights(w, want_w, 3 * bound, m.lens)
    close_out(m, run(m), want)


PAIRS = {   # more than two waves of score tiles: blocks of query rows x tiles of 256 tokens > 296
    "f16-5-blocks": dict(prefix=15800, lens=(3, 0, 130) * 6, H=32, r=128),   # the last pair's second CTA has no rows
    "f16-2-blocks": dict(prefix=38000, lens=(5, 9), H=100, r=64),
    "f16-heads-6": dict(prefix=26001, lens=(2,) * 50, H=6, r=192),
    "bf16": dict(cache="bf16", weight="bf16", out="bf16", prefix=19001, lens=(1,) * 16, H=32, r=192),
    "i8": dict(cache="i8", prefix=19999, lens=(20,) * 16, H=32, r=256),
    "i4": dict(cache="i4", prefix=25600, lens=(0, 7, 20) * 3, H=32, r=128),
    "rope": dict(prefix=15900, lens=(3, 0, 130) * 6, H=32, d_h=128, r=128, rope=True),
}


@pytest.mark.parametrize("name", list(PAIRS))
def test_cta_pairs_against_the_definition(cuda_ok, name):
    form = PAIRS[name]
    m = Layer(**form)
    tiles, blocks = -(-form["prefix"] // 256), -(-m.B // min(m.B, 128 // m.H))
    assert blocks > 1 and tiles * blocks > 2 * torch.cuda.get_device_properties(0).multi_processor_count
    want, want_w, bound = m.exact()
    w = torch.zeros(m.B, m.max_len, device=DEV)
    close_out(m, run(m, weights=w), want)
    close_weights(w, want_w, 3 * bound, m.lens)
