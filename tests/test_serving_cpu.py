"""Host-side refusals of the serving calls (no GPU: the pointers are never
dereferenced) and the order of the eviction's weight keys."""
import ctypes

import numpy as np
import pytest

import rank_joint_qkv_b200 as q

OK = 1 << 20   # an aligned address


def dims(**kw):
    base = dict(E=512, H=4, d_h=128, r=256, batch=2, max_len=300)
    base.update({k: kw.pop(k) for k in list(kw) if k in base})
    return q.make_dims(*(base[k] for k in ("E", "H", "d_h", "r", "batch", "max_len")), **kw)


def refused(call, status, words):
    st = call()
    assert st == status, (st, q._lib.qsvd_last_error())
    assert words in q._lib.qsvd_last_error().decode()


def weights_call(d, ws_bytes=None, workspace=OK, weights=OK + 4096, cache=OK, scales=None, lengths=OK, out=OK, qin=OK,
                 packed=OK, splits=4):
    n = ctypes.c_size_t(q.decode_weights_workspace_bytes(d, splits) if ws_bytes is None else ws_bytes)
    p = lambda v: None if v is None else ctypes.c_void_p(v)  # noqa: E731
    return lambda: q._lib.qsvd_decode_attn_weights(ctypes.byref(d), p(packed), p(qin), 1, p(cache), p(scales), p(lengths),
                                                   splits, p(workspace), ctypes.byref(n), p(out), p(weights), 1, None)


def test_weights_workspace_has_room_for_the_scores():
    d = dims()
    scores = 2 * 4 * 300 * 4   # B x H x max_len
    assert q.decode_weights_workspace_bytes(d, 4) >= q.decode_workspace_bytes(d, 4) + scores
    r = dims(rope=True)        # the rotary decode keeps its scores in any case
    assert q.decode_weights_workspace_bytes(r, 4) - q.decode_workspace_bytes(r, 4) < scores


def test_weights_refusals():
    d = dims()
    bad, ws = q.QSVD_ERR_INVALID_ARG, q.QSVD_ERR_WORKSPACE
    refused(weights_call(d, weights=None), bad, "weights must be given")
    refused(weights_call(d, weights=OK + 2), bad, "4-byte aligned")
    refused(weights_call(d, ws_bytes=q.decode_workspace_bytes(d, 4)), ws, "workspace holds")
    refused(weights_call(d, cache=None), bad, "cache is NULL")
    refused(weights_call(d, lengths=None), bad, "NULL")
    refused(weights_call(d, cache=OK + 8), bad, "16-byte aligned")
    refused(weights_call(dims(cache="i8")), bad, "int caches need scales")
    refused(weights_call(dims(), splits=4, out=None), bad, "out is NULL")
    x = dims(kernel=q.QSVD_KERNEL_TCGEN05_CTA, r=96)
    with pytest.raises(q.QsvdError) as e:
        q.decode_weights_workspace_bytes(x, 4)
    assert e.value.status == q.QSVD_ERR_UNSUPPORTED
    with pytest.raises(q.QsvdError) as e:
        q.decode_weights_workspace_bytes(d, -1)
    assert e.value.status == bad


def evict_call(d, budget=64, sink=4, recent=16, ws_bytes=None, workspace=OK, weights=OK, lengths=OK, cache=OK,
               scales=None, dst_max_len=300, dst_cache=OK, dst_scales=None, dst_weights=OK, dst_lengths=OK, kept=None):
    n = ctypes.c_size_t((1 << 30) if ws_bytes is None else ws_bytes)
    p = lambda v: None if v is None else ctypes.c_void_p(v)  # noqa: E731
    return lambda: q._lib.qsvd_evict_rows(ctypes.byref(d), p(weights), p(lengths), budget, sink, recent, p(cache),
                                          p(scales), dst_max_len, p(dst_cache), p(dst_scales), p(dst_weights),
                                          p(dst_lengths), p(kept), None, p(workspace), ctypes.byref(n), None)


def test_evict_refusals():
    d = dims()
    bad = q.QSVD_ERR_INVALID_ARG
    far = OK + (1 << 30)
    for budget in (0, -1, 301):
        refused(evict_call(d, budget=budget), bad, "budget")
    refused(evict_call(d, sink=-1), bad, "sink")
    refused(evict_call(d, recent=-1), bad, "recent")
    refused(evict_call(d, sink=40, recent=30), bad, "within the budget")
    refused(evict_call(d, sink=0x7FFFFFFF, recent=0x7FFFFFFF), bad, "within the budget")   # no 32-bit wrap
    refused(evict_call(d, dst_max_len=63, dst_cache=far), bad, "at least the budget")
    refused(evict_call(d, dst_max_len=1 << 30, dst_cache=far), bad, "below 2^31")
    refused(evict_call(d, ws_bytes=q.evict_workspace_bytes(d, 64) - 1), q.QSVD_ERR_WORKSPACE, "workspace holds")
    for k in ("weights", "lengths", "cache", "dst_cache", "dst_lengths"):
        refused(evict_call(d, **{k: None}), bad, "NULL")
    for k in ("cache", "dst_cache", "workspace"):
        refused(evict_call(d, **{k: OK + 8}), bad, "16-byte aligned")
    for k in ("weights", "lengths", "dst_weights", "dst_lengths", "kept"):
        refused(evict_call(d, **{k: OK + 2}), bad, "4-byte aligned")
    i8 = dims(cache="i8")
    refused(evict_call(i8), bad, "need scales")
    refused(evict_call(i8, scales=OK + 1, dst_scales=OK + 1), bad, "2-byte")
    # overlap: in place with another capacity, or a destination inside its source
    refused(evict_call(d, dst_max_len=100), bad, "or not overlap")
    refused(evict_call(d, dst_cache=OK + 512), bad, "or not overlap")
    refused(evict_call(d, dst_cache=OK - 512), bad, "or not overlap")
    refused(evict_call(d, dst_cache=far, dst_weights=OK + 64), bad, "or not overlap")
    refused(evict_call(d, dst_cache=far, dst_weights=far, dst_lengths=OK + 4), bad, "or not overlap")
    refused(evict_call(i8, scales=OK, dst_scales=OK + 2), bad, "or not overlap")


def test_weight_keys_keep_the_order():
    """The integer keys of evict.cu (restated): ascending with the weight, -0 equal to 0, NaN below everything."""
    def key(w):
        w = np.asarray(w, np.float32)
        u = np.where(w == 0, np.float32(0), w).view(np.uint32)
        k = np.where(u & 0x80000000, ~u, u | 0x80000000).astype(np.uint32)
        return np.where(np.isnan(w), np.uint32(0), k)
    w = np.array([-np.inf, -3.4e38, -1.0, -1e-45, 0.0, 1e-45, 1e-38, 0.5, 1.0, 3.4e38, np.inf], np.float32)
    k = key(w).astype(np.int64)
    assert (np.diff(k) > 0).all() and k[0] > 0
    assert key([np.nan, -np.nan]).tolist() == [0, 0] and key([-0.0]) == key([0.0])
    src = open(q.LIB_PATH.replace("libqsvd.so", "csrc/evict.cu")).read()
    assert "return (u & 0x80000000u) ? ~u : (u | 0x80000000u);" in src and "if (isnan(w)) return 0u;" in src


def shared_call(d, plen=100, splits=4, prefix=OK, prefix_scales=None, workspace=OK, ws_bytes=1 << 40, weights=None, cache=OK,
                scales=None, out=OK, qin=OK, packed=OK, lengths=OK):
    n = ctypes.c_size_t(ws_bytes)
    p = lambda v: None if v is None else ctypes.c_void_p(v)  # noqa: E731
    return lambda: q._lib.qsvd_decode_attn_shared(ctypes.byref(d), p(packed), p(qin), 1, p(prefix), p(prefix_scales), plen,
                                                  p(cache), p(scales), p(lengths), splits, p(workspace), ctypes.byref(n),
                                                  p(out), p(weights), 1, None)


def test_shared_refusals():
    d = dims()
    bad = q.QSVD_ERR_INVALID_ARG
    refused(shared_call(dims(rope=True, batch=1), plen=0x7FFFFFFF), bad, "max_len + prefix_len")
    refused(shared_call(d, plen=-1), bad, "prefix_len")
    refused(shared_call(d, plen=1 << 30), bad, "below 2^31")
    refused(shared_call(d, prefix=None), bad, "prefix must be given")
    refused(shared_call(d, prefix=OK + 8), bad, "16-byte aligned")
    refused(shared_call(dims(cache="i8"), scales=OK), bad, "prefix_scales")
    refused(shared_call(dims(cache="i8"), scales=OK, prefix_scales=OK + 1), bad, "2-byte")
    refused(shared_call(dims(cache="i8"), prefix_scales=OK), bad, "int caches need scales")
    refused(shared_call(d, weights=OK + 1), bad, "4-byte aligned")
    refused(shared_call(d, ws_bytes=q.decode_shared_workspace_bytes(d, 100, 4) - 1), q.QSVD_ERR_WORKSPACE, "workspace holds")
    for k in ("cache", "lengths", "packed", "qin", "out"):
        refused(shared_call(d, **{k: None}), bad, "NULL")
    refused(shared_call(d, splits=-1), bad, "num_splits")
    refused(shared_call(dims(d_h=24, H=8, E=192, r=128, out_proj="chain")), q.QSVD_ERR_UNSUPPORTED, "output projection")
    assert q.decode_shared_workspace_bytes(d, 0, 4) < q.decode_shared_workspace_bytes(d, 1, 4)
