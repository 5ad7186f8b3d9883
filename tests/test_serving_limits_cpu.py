"""The serving calls at the largest sizes their 32-bit counts allow (host side, no GPU)."""
import pytest

import rank_joint_qkv_b200 as q
from tests.test_serving_cpu import refused, shared_call


def test_the_longest_prefix():
    """Rows of scores are padded to 256 tokens: past 2^31 - 256 the padded length does not fit 32 bits."""
    d = q.make_dims(64, 1, 64, 64, 1, 8, cache="f16")
    most = 2 ** 31 - 256
    p_bytes = 128 * most * 2   # a block of 128 query rows of P
    assert p_bytes < q.decode_shared_workspace_bytes(d, most, 1) < 1.1 * p_bytes
    for n in (most + 1, 2 ** 31 - 1):
        refused(shared_call(d, plen=n, splits=1), q.QSVD_ERR_INVALID_ARG, "2^31 - 256")
        with pytest.raises(q.QsvdError):
            q.decode_shared_workspace_bytes(d, n, 1)


def test_sizes_of_the_largest_batches():
    assert q.decode_shared_workspace_bytes(q.make_dims(64, 1, 64, 64, 65535, 8, cache="f16"), 32767, 1) > 2 ** 32
    d = q.make_dims(64, 1, 64, 64, 1, 2 ** 31 - 1, cache="i4", group=32)
    assert q.decode_weights_workspace_bytes(d, 1) > 4 * (2 ** 31 - 1)
    assert q.evict_workspace_bytes(d, 2 ** 31 - 1) > 4 * (2 ** 31 - 1)
