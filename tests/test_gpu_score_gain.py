"""The gain on the query of the serving calls, which makes up for what the tensor cores' accumulators cut off: how far the
scores are from themselves, fitted from float32 attention weights.

If the own rows' scores s were (1 + x) s and the prefix's (1 + y) s, a weight w_t = sum_h p_{h,t} would move by
  x sum_h p_{h,t} (s_{h,t} - sum_{own u} p_{h,u} s_{h,u}) - y sum_h p_{h,t} sum_{prefix u} p_{h,u} s_{h,u}
to first order; x and y come out of a least-squares fit over all rows.  Without the gain x is -(0.9 a + 1.4 b) 2^-25 for dense
rows, a the accumulations of a score (r / 16; on a prefix once per part of the query) and b those of the projections; the gain
must take at least half of that off.  On CUDA cores and for int8 rows a is 0.  Beside that 2^-22: a weight's float32 error of
2^-20 at most (exponential, reciprocal, sums) averaged over a thousand rows, against scores of some units."""
import pytest
import torch

import rank_joint_qkv_b200 as q
from tests.serving_util import DEV, Layer

pytestmark = pytest.mark.gpu

A, S, T, C = (q.QSVD_KERNEL_AUTO, q.QSVD_KERNEL_SIMT, q.QSVD_KERNEL_TCGEN05_CTA, q.QSVD_KERNEL_TCGEN05_CLUSTER)
DENSE = dict(H=4, d_h=128, r=1536, lens=(600, 400, 33), peak=3.0)
CASES = {   # layer, accumulations of an own score and of a prefix's
    "f16": (dict(DENSE, kernel=T), 96, 0),
    "f16-r2560": (dict(DENSE, r=2560, kernel=T), 160, 0),
    "bf16": (dict(DENSE, cache="bf16", weight="bf16", kernel=T), 96, 0),
    "f16-cluster": (dict(DENSE, kernel=C), 16, 0),   # 256 channels a CTA
    "i8": (dict(DENSE, cache="i8", kernel=T), 0, 0),
    "f16-simt": (dict(DENSE, kernel=S), 0, 0),
    "f16-rope": (dict(DENSE, rope=True), 96, 0),
    "f16-prefix": (dict(DENSE, prefix=900), 96, 192),
    "bf16-prefix": (dict(DENSE, cache="bf16", weight="bf16", prefix=900), 96, 288),
    "i8-prefix": (dict(DENSE, cache="i8", prefix=900), 0, 288),
    "f16-rope-prefix": (dict(DENSE, rope=True, prefix=900), 96, 96),
    "f16-simt-prefix": (dict(DENSE, kernel=S, prefix=900), 0, 0),
    # own rows on the tensor cores, the prefix on the CUDA cores
    "f16-rope-130-heads": (dict(H=130, d_h=128, r=1472, lens=(200, 33), peak=3.0, rope=True, prefix=150), 92, 0),
}


def shares(m):
    """Per own row of the batch: w, the coefficient of x and of y, as above."""
    wq, wk = m.wuq.double(), m.wuk.double()
    H, d_h, P = m.H, m.d_h, m.prefix_values.shape[0]
    out = []
    for b, n in enumerate(m.lens):
        c = torch.cat([m.prefix_values, m.values[b, :n]])
        qb, k = (m.qin[b].double() @ wq).view(H, d_h), (c @ wk).view(-1, H, d_h)
        if m.rope:
            ang = torch.arange(P + n, device=DEV, dtype=torch.float64)[:, None] * \
                torch.pow(10000.0, -2.0 * torch.arange(d_h // 2, device=DEV, dtype=torch.float64) / d_h)
            spin = torch.polar(torch.ones_like(ang), ang)
            pairs = lambda x: torch.complex(x[..., :d_h // 2], x[..., d_h // 2:])  # noqa: E731
            s = ((pairs(k) * spin[:, None]) * (pairs(qb) * spin[P + n - 1]).conj()).real.sum(-1) * d_h ** -0.5
        else:
            s = torch.einsum("thd,hd->th", k, qb) * d_h ** -0.5
        p = torch.softmax(s, 0)
        own, ahead = (p[P:] * s[P:]).sum(0), (p[:P] * s[:P]).sum(0)
        out.append(torch.stack([p[P:].sum(1), (p[P:] * (s[P:] - own)).sum(1), -(p[P:] * ahead).sum(1)], 1))
    return torch.cat(out)


@pytest.mark.parametrize("name", list(CASES))
def test_scores_are_right_on_the_mean(cuda_ok, name):
    form, own, ahead = CASES[name]
    m = Layer(seed=4, **form)
    P = m.prefix_values.shape[0]
    w, out = torch.zeros(m.B, m.max_len, device=DEV), m.empty_out()
    q.qsvd_decode_attn_shared(m.dims, m.packed, m.qin, True, m.prefix, m.prefix_scales, P, m.cache, m.scales, m.lengths, out,
                              weights=w, accumulate=False)
    w_, cx, cy = shares(m).unbind(1)
    got = torch.cat([w[b, :n].double() for b, n in enumerate(m.lens)])
    cols = torch.stack([cx, cy] if P else [cx], 1) / w_[:, None]
    x = torch.linalg.lstsq(cols.cpu(), ((got - w_) / w_)[:, None].cpu()).solution[:, 0].tolist()
    projections = (min(32, m.r // 16) + 3) // 4 + (0 if m.rope else m.d_h // 16)
    for off, steps in zip(x, (own, ahead)):
        short = (0.9 * steps + 1.4 * projections) * 2.0 ** -25
        print(name, "off by %.2e, %.2e without a gain" % (off, -short))
        assert abs(off) <= short / 2 + 2.0 ** -22


def test_a_score_of_few_terms_is_at_most_the_gain_too_large(cuda_ok):
    """Two channels of 1536 a row, one sign: nearly nothing is cut off, so the score is too large by up to the gain
    (0.9 x 96 + 1.4 x 4) 2^-25; two fp16 parts of the query 2^-22, its three products and sums 2^-23 each, 2^-20 for the weights."""
    B, n, r, d_h = 4, 300, 1536, 64
    g = torch.Generator()
    g.manual_seed(5)
    a = (1 + torch.rand(r, generator=g)).half().double()
    rows = torch.zeros(n, r, dtype=torch.float64)
    for t in range(1, n):
        rows[t, torch.randperm(r, generator=g)[:2]] = (16 * torch.rand(2, generator=g)).half().double()
    query = (1 + torch.rand(B, generator=g)).float()
    dims = q.make_dims(d_h, 1, d_h, r, B, n, cache="f16", weight="f16", kernel=T)
    wuk = torch.zeros(r, d_h, dtype=torch.float64)
    wuk[:, 0] = a
    z = torch.zeros(r, d_h, device=DEV, dtype=torch.float16)
    packed = q.qsvd_prepare_weights(dims, z.t().contiguous(), z, wuk.half().to(DEV), z)
    qin = torch.zeros(B, d_h)
    qin[:, 0] = query
    cache = rows.half()[None].repeat(B, 1, 1).contiguous().to(DEV)
    w, out = torch.zeros(B, n, device=DEV), torch.zeros(B, d_h, device=DEV)
    q.qsvd_decode_attn_weights(dims, packed, qin.to(DEV), False, cache, None,
                               torch.full((B,), n, dtype=torch.int32, device=DEV), out, w, accumulate=False)
    scores = query.double()[:, None] * (rows @ a)[None] / d_h ** 0.5
    got = w.double().cpu()
    off = (got[:, 1:] / got[:, :1]).log() - scores[:, 1:]
    lim = ((0.9 * 96 + 1.4 * 4) * 2.0 ** -25 + 2.0 ** -22 + 3 * 2.0 ** -23) * scores[:, 1:] + 2.0 ** -20
    assert float((off.abs() / lim).max()) <= 1.0


# bf16 weights take a third part of the activations, an int8 prefix a second pass over its rows, both behind the others
LATER_PARTS = {"bf16": dict(cache="bf16", weight="bf16", r=512), "bf16-r256": dict(cache="bf16", weight="bf16", r=256),
               "f16-rows": dict(weight="bf16", r=512), "i8": dict(cache="i8", weight="bf16", r=1536),
               "i8-prefix": dict(cache="i8", r=1536, prefix=900), "bf16-prefix": dict(cache="bf16", weight="bf16", r=1536, prefix=900)}


@pytest.mark.parametrize("name", list(LATER_PARTS))
def test_parts_that_are_multiplied_behind_others(cuda_ok, name):
    """Accumulations onto a sum of its full size lose more.  Left out they are 8 and 8 (the projections') x 0.86 x 2^-25 =
    4.1e-7, or 96 x 0.14 x 2^-25 = 4e-7 of an int8 prefix; the mean of five inputs, each known to 1.4e-7 or better (the
    spread of the fits), has to be within 2^-22 = 2.4e-7."""
    off = []
    for seed in range(5):
        m = Layer(seed=seed, H=4, d_h=128, lens=(600, 400, 60), **LATER_PARTS[name])
        P = m.prefix_values.shape[0]
        w, out = torch.zeros(m.B, m.max_len, device=DEV), m.empty_out()
        q.qsvd_decode_attn_shared(m.dims, m.packed, m.qin, True, m.prefix, m.prefix_scales, P, m.cache, m.scales, m.lengths,
                                  out, weights=w, accumulate=False)
        w_, cx, cy = shares(m).unbind(1)
        got = torch.cat([w[b, :n].double() for b, n in enumerate(m.lens)])
        cols = torch.stack([cx, cy] if P else [cx], 1) / w_[:, None]
        off.append(torch.linalg.lstsq(cols.cpu(), ((got - w_) / w_)[:, None].cpu()).solution[:, 0])
    off = torch.stack(off).mean(0)
    print(name, off.tolist())
    assert float(off.abs().max()) <= 2.0 ** -22
