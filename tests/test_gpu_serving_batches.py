"""The serving calls on thousands of sequences, up to the most a call takes."""
import pytest
import torch

import rank_joint_qkv_b200 as q
from tests.serving_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [3001, 65535])
@pytest.mark.parametrize("prefix", [0, 300])
def test_many_sequences(cuda_ok, B, prefix):
    """One head, a few own rows each; decode with weights, then a cut to two rows, against batched float64.  A score's bound:
    two fp16 parts of the query and of the absorbed one (2^-22 each), float32 sums of 64 terms, twice as many accumulations on
    the prefix, all below 2^-16 of the sum of magnitudes; an output adds the rounding of P, 2^-11, and the two parts of the
    merged latent."""
    d_h = r = 64
    max_len, budget = 5, 2
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    dims = q.make_dims(d_h, 1, d_h, r, B, max_len, cache="f16", weight="f16")
    wuq, wuk, wuv = ((rnd(r, d_h) / 8).half() for _ in range(3))
    packed = q.qsvd_prepare_weights(dims, wuq.t().contiguous(), wuq, wuk, wuv)
    cache, pre, qin = rnd(B, max_len, r).half(), rnd(max(prefix, 1), r).half()[:prefix], rnd(B, r)
    lengths = (torch.arange(B, device=DEV) % (max_len + 1)).int()
    out, w = torch.zeros(B, d_h, device=DEV), torch.zeros(B, max_len, device=DEV)
    ws = q.qsvd_decode_attn_shared(dims, packed, qin, True, pre if prefix else None, None, prefix, cache, None, lengths, out,
                                   weights=w, accumulate=False)
    torch.cuda.synchronize()
    assert q.status_word(ws) == 0
    f = lambda x: x.double()  # noqa: E731
    qq, wk, wv = f(qin) @ f(wuq), f(wuk), f(wuv)
    live = torch.arange(max_len, device=DEV)[None] < lengths[:, None]
    own = torch.einsum("btr,br->bt", f(cache), qq @ wk.t()) / 8
    mags = torch.einsum("btr,br->bt", f(cache).abs(), f(qin).abs() @ f(wuq).abs() @ wk.abs().t()).max() / 8
    s = torch.cat([(qq @ wk.t()) @ f(pre).t() / 8, own.masked_fill(~live, -torch.inf)], 1)
    p = torch.softmax(s, 1).nan_to_num(0.0)   # no rows at all: zeros
    v = torch.cat([(f(pre) @ wv)[None].expand(B, -1, -1), torch.einsum("btr,rd->btd", f(cache), wv)], 1) if B < 5000 else None
    want_w = p[:, prefix:]
    bound = float(mags) * 2.0 ** -16
    assert bool(((f(w) - want_w).abs() <= (2.2 * bound + 2.0 ** -18) * want_w).all())
    if v is not None:
        want, spread = torch.einsum("bt,btd->bd", p, v), torch.einsum("bt,btd->bd", p, v.abs())
        assert bool(((f(out) - want).abs() <= (2.2 * bound + 2.0 ** -11 + 2.0 ** -14) * spread + 1e-6).all())
    # a cut in place: the two heaviest of three to five rows, in order
    kept = torch.zeros(B, budget, dtype=torch.int32, device=DEV)
    rows, weights, lens = cache.clone(), w.clone(), lengths.clone()
    q.qsvd_evict_rows(dims, weights, lens, budget, rows, kept=kept)
    torch.cuda.synchronize()
    key = torch.where(live, w, -1.0)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :budget]
    at = torch.where(lengths[:, None] > budget, order, torch.arange(budget, device=DEV)[None]).sort(1).values
    there = torch.arange(budget, device=DEV)[None] < lengths[:, None]
    assert torch.equal(kept, torch.where(there, at, -1).int()) and torch.equal(lens, lengths.clamp(max=budget))
    moved = torch.gather(cache, 1, at[..., None].expand(-1, -1, r))
    assert torch.equal(rows[:, :budget][there], moved[there])
    assert torch.equal(weights[:, :budget], torch.where(there, torch.gather(w, 1, at), 0.0)) and not weights[:, budget:].any()
