"""Rotary decode at every head size it takes (multiples of 64 up to 256), on the CUDA cores: the plain step, the rows'
weights and a shared prefix against the definition in 64 bits."""
import pytest
import torch

import rank_joint_qkv_b200 as q
from tests.serving_util import DEV, Layer, close_weights, rel_err

pytestmark = pytest.mark.gpu

FORMS = [dict(cache="f32", weight="f32", r=64), dict(cache="f16", weight="f16", r=96),
         dict(cache="bf16", weight="bf16", r=128), dict(cache="i8", weight="f16", r=128)]


@pytest.mark.parametrize("prefix", [0, 37])
@pytest.mark.parametrize("d_h", [64, 128, 192, 256])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: f["cache"])
def test_against_the_definition(cuda_ok, form, d_h, prefix):
    m = Layer(H=3, d_h=d_h, rope=True, lens=(40, 0, 17, 130), prefix=prefix, kernel=q.QSVD_KERNEL_SIMT, **form)
    want, want_w, bound = m.exact()
    out, w = m.empty_out(), torch.zeros(m.B, m.max_len, device=DEV)
    q.qsvd_decode_attn_shared(m.dims, m.packed, m.qin, True, m.prefix, m.prefix_scales, prefix, m.cache, m.scales, m.lengths,
                              out, weights=w, accumulate=False)
    torch.cuda.synchronize()
    # float32 sums of r, d_h and 167 terms of a float32 table: 1e-4 of rms for float32 rows, the decode's 2e-3 otherwise
    assert torch.isfinite(out).all() and rel_err(out, want) <= (1e-4 if form["cache"] == "f32" else 2e-3)
    close_weights(w, want_w, 3 * bound, m.lens)
    if prefix == 0:
        plain = m.empty_out()
        q.qsvd_decode_attn(m.dims, m.packed, m.qin, True, m.cache, m.scales, m.lengths, plain)
        torch.cuda.synchronize()
        assert rel_err(plain, want) <= (1e-4 if form["cache"] == "f32" else 2e-3)
