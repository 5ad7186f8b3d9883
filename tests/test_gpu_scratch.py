"""Calls without a workspace on two streams at once: each takes its own scratch."""
import pytest
import torch

import rank_joint_qkv_b200 as q
from tests.serving_util import DEV, Layer

pytestmark = pytest.mark.gpu


def calls():
    """name -> (call(out, stream), outputs) on inputs that nothing changes."""
    m = Layer(prefix=600, lens=(40, 0, 333), H=8)
    weights = torch.rand(m.B, m.max_len, device=DEV)
    budget = 64

    def shared(o, s):
        q.qsvd_decode_attn_shared(m.dims, m.packed, m.qin, True, m.prefix, None, 600, m.cache, None, m.lengths, o[0], stream=s)

    def with_weights(o, s):
        q.qsvd_decode_attn_weights(m.dims, m.packed, m.qin, True, m.cache, None, m.lengths, o[0], o[1], accumulate=False, stream=s)

    def decode(o, s):
        q.qsvd_decode_attn(m.dims, m.packed, m.qin, True, m.cache, None, m.lengths, o[0], stream=s)

    def evict(o, s):
        q.qsvd_evict_rows(m.dims, weights, m.lengths, budget, m.cache, sink=2, recent=8, dst_max_len=budget, dst_cache=o[0],
                          dst_weights=o[1], dst_lengths=o[2], stream=s)

    out = lambda: [m.empty_out()]  # noqa: E731
    return {"shared": (shared, out), "decode": (decode, out),
            "weights": (with_weights, lambda: [m.empty_out(), torch.zeros(m.B, m.max_len, device=DEV)]),
            "evict": (evict, lambda: [torch.zeros(m.B, budget, m.r, dtype=m.cache.dtype, device=DEV),
                                      torch.zeros(m.B, budget, device=DEV),
                                      torch.zeros(m.B, dtype=torch.int32, device=DEV)])}


@pytest.mark.parametrize("held", ["current", "side"])
@pytest.mark.parametrize("name", ["shared", "decode", "weights", "evict"])
def test_a_held_stream_keeps_its_scratch(cuda_ok, name, held):
    """One stream is held up, calls are queued on both, and every returned scratch is dropped at once."""
    call, outputs = calls()[name]
    want = outputs()
    call(want, None)
    side = torch.cuda.Stream()
    order = [None, side] if held == "current" else [side, None]
    outs = [outputs() for _ in range(12)]
    torch.cuda.synchronize()
    for i in range(0, len(outs), 2):
        if held == "current":
            torch.cuda._sleep(2_000_000)
        else:
            with torch.cuda.stream(side):
                torch.cuda._sleep(2_000_000)
        for o, s in zip(outs[i:i + 2], order):
            call(o, s)
    torch.cuda.synchronize()
    for o in outs:
        for x, w in zip(o, want):
            assert torch.equal(x, w)
