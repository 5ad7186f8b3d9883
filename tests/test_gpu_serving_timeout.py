"""The serving calls beside a wait that runs out in the own rows' split kernel: the call returns with the status bit, the
prefix's and the eviction's kernels run to their end, and the next call on the same workspace is exact again."""
import pytest
import torch

import rank_joint_qkv_b200 as q
from tests.serving_util import DEV, Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", [dict(H=8), dict(H=8, cache="bf16", weight="bf16"), dict(H=32, cache="i8"),
                                  dict(H=8, prefix=0)], ids=["f16", "bf16", "i8", "weights"])
def test_expired_wait_is_flagged_and_the_next_call_exact(cuda_ok, form):
    form = dict(dict(prefix=1100, lens=(40, 0, 333), kernel=q.QSVD_KERNEL_TCGEN05_CTA), **form)
    m = Layer(**form)
    P = form["prefix"]
    ws = torch.empty(q.decode_shared_workspace_bytes(m.dims, P), dtype=torch.uint8, device=DEV)

    def run():
        out, w = m.empty_out(), torch.zeros(m.B, m.max_len, device=DEV)
        q.qsvd_decode_attn_shared(m.dims, m.packed, m.qin, True, m.prefix, m.prefix_scales, P, m.cache, m.scales, m.lengths,
                                  out, weights=w, accumulate=False, workspace=ws)
        torch.cuda.synchronize()
        return out, w, q.status_word(ws)

    want = run()
    assert want[2] == 0
    q.qsvd_testing_set_score_wait_ns(200_000)
    try:
        assert run()[2] & q.QSVD_STATUS_TIMEOUT
    finally:
        q.qsvd_testing_set_score_wait_ns(0)
    again = run()
    assert again[2] == 0 and torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
