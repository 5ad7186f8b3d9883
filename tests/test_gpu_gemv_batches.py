"""The projections of large batches: a sequence's output does not depend on how many others there are, whichever way the
blocks of 16 sequences and the sums of the k-splits are laid out on the GPU."""
import pytest
import torch

import rank_joint_qkv_b200 as q
from tests.serving_util import DEV, Layer

pytestmark = pytest.mark.gpu

# k-splits of the query and value projections (r / 512) and of the output projection (E / 512)
FORMS = {
    "1": dict(H=8, d_h=64, r=256),
    "2-and-4": dict(H=16, d_h=128, r=768, out_proj="chain"),
    "3": dict(H=32, d_h=64, r=1280),
    "3-bf16": dict(H=32, d_h=64, r=1280, cache="bf16", weight="bf16"),
    "2-and-5": dict(H=20, d_h=128, r=640, out_proj="chain"),
    "5": dict(H=40, d_h=64, r=2304),
    "1-and-8": dict(H=32, d_h=128, r=256, out_proj="chain"),
    "9": dict(H=8, d_h=64, r=4160),
}


@pytest.mark.parametrize("B", [15, 33, 50, 64, 130, 500])
@pytest.mark.parametrize("name", list(FORMS))
def test_a_row_is_the_same_in_any_batch(cuda_ok, name, B):
    m = Layer(lens=[1 + 7 * b % 60 for b in range(B)], seed=2, **FORMS[name])   # one tile a sequence, in one split
    if m.dims.out_proj:
        g = torch.Generator(device=DEV)
        g.manual_seed(3)
        wo = (torch.randn(m.E, m.E, generator=g, device=DEV) / m.E ** 0.5).to(m.wuq.dtype)
        q.qsvd_prepare_out_proj(m.dims, wo, m.packed)
    out, w = m.empty_out(), torch.zeros(B, m.max_len, device=DEV)
    q.qsvd_decode_attn(m.dims, m.packed, m.qin, True, m.cache, None, m.lengths, out)
    shared = m.empty_out()
    q.qsvd_decode_attn_weights(m.dims, m.packed, m.qin, True, m.cache, None, m.lengths, shared, w, accumulate=False)
    x = torch.randn(B, m.E, device=DEV).to(m.wd.dtype)
    c = torch.zeros(B, m.r, device=DEV)
    q.qsvd_append_latent(m.dims, m.packed, x, m.lengths, m.cache, None, c)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()
    one = q.make_dims(m.E, m.H, m.d_h, m.r, 1, m.max_len, cache="bf16" if m.cache.dtype == torch.bfloat16 else "f16",
                      weight=m.weight, out_proj=FORMS[name].get("out_proj"))
    for b in sorted({0, 1, B // 2, 16 * (B // 16) - 1, B - 1} & set(range(B))):
        o1, w1 = torch.zeros(1, m.E, device=DEV), torch.zeros(1, m.max_len, device=DEV)
        args = (one, m.packed, m.qin[b:b + 1].contiguous(), True, m.cache[b:b + 1], None, m.lengths[b:b + 1].clone())
        q.qsvd_decode_attn(*args, o1)
        assert torch.equal(o1[0], out[b])
        q.qsvd_decode_attn_weights(*args, o1, w1, accumulate=False)
        assert torch.equal(o1[0], shared[b]) and torch.equal(w1[0], w[b])
        c1, row = torch.zeros(1, m.r, device=DEV), m.cache[b:b + 1].clone()
        q.qsvd_append_latent(one, m.packed, x[b:b + 1].contiguous(), m.lengths[b:b + 1].clone(), row, None, c1)
        assert torch.equal(c1[0], c[b])
