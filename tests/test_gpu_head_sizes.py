"""Decode with head sizes that do not divide 128 rows of the value
up-projection evenly over the combine's k-splits (256 / d_h of them)."""
import pytest

import rank_joint_qkv_b200 as q
from tests.serving_util import Layer, rel_err

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d_h", [8, 24, 40, 48, 72, 80, 120, 200, 256])
@pytest.mark.parametrize("cache,weight,bar", [("f32", "f32", 1e-4), ("f16", "f16", 2e-3)])
def test_decode_output(cuda_ok, d_h, cache, weight, bar):
    """fp32 rows 1e-4, 16-bit rows 2e-3 of rms (the decode's bars); CUDA-core split kernel, so P is not rounded."""
    m = Layer(cache=cache, weight=weight, H=8, d_h=d_h, r=160, lens=(200, 3, 129), kernel=q.QSVD_KERNEL_SIMT)
    out = m.empty_out()
    q.qsvd_decode_attn(m.dims, m.packed, m.qin, True, m.cache, m.scales, m.lengths, out)
    assert rel_err(out, m.exact()[0]) <= bar


@pytest.mark.parametrize("r", [512, 544, 1024, 4096, 4128])
@pytest.mark.parametrize("batch", [1, 17, 50])
@pytest.mark.parametrize("weight", ["f16", "bf16"])
def test_decode_output_at_projection_splits(cuda_ok, r, batch, weight):
    """One to nine k-splits of the projections' GEMV (512 rows each; up to eight in a cluster), and blocks of 16
    sequences walked by one CTA."""
    m = Layer(cache=weight, weight=weight, H=4, d_h=64, r=r, lens=tuple(1 + 7 * i % 40 for i in range(batch)),
              kernel=q.QSVD_KERNEL_SIMT)
    out = m.empty_out()
    q.qsvd_decode_attn(m.dims, m.packed, m.qin, True, m.cache, m.scales, m.lengths, out)
    assert rel_err(out, m.exact()[0]) <= 2e-3
