"""Refusals of the entry points between the linear layers, on the host: the
pointers are fake and no call here gets past the argument checks (or it is a
no-op, or it stops at the device check where there is no device)."""
import ctypes

import pytest
import torch

import weight_only_bit_awq_b200 as awq

L = awq.lib
A, B, C, D, E, F, G, H = (0x7F0000000000 + (i << 36) for i in range(8))


def _norm(x=A, residual=B, w=C, eps=1e-5, h=D, y=E, M=4, K=256):
    return L.awq_rmsnorm(x, residual, w, eps, h, y, M, K, None)


def _norm8(x=A, residual=B, w=C, eps=1e-5, h=D, x8=E, sx=F, M=4, K=256):
    return L.awq_rmsnorm_fp8(x, residual, w, eps, h, x8, sx, M, K, None)


@pytest.mark.parametrize("fn", [_norm, _norm8])
def test_rmsnorm_refusals(fn):
    assert fn(M=-1) == awq.AWQ_ERR_SHAPE
    assert fn(K=0) == awq.AWQ_ERR_SHAPE
    assert fn(K=250) == awq.AWQ_ERR_SHAPE
    assert fn(K=(1 << 22) + 8) == awq.AWQ_ERR_UNSUPPORTED
    assert fn(M=(1 << 24) + 1) == awq.AWQ_ERR_UNSUPPORTED
    assert fn(x=None) == awq.AWQ_ERR_INVALID_ARG
    assert fn(w=None) == awq.AWQ_ERR_INVALID_ARG
    assert fn(h=None) == awq.AWQ_ERR_INVALID_ARG             # a residual needs h
    assert fn(residual=None) == awq.AWQ_ERR_INVALID_ARG      # and h a residual
    for eps in (-1e-5, float("nan"), float("inf")):
        assert fn(eps=eps) == awq.AWQ_ERR_INVALID_ARG
    assert fn(x=A + 8) == awq.AWQ_ERR_ALIGNMENT
    assert fn(residual=B + 2) == awq.AWQ_ERR_ALIGNMENT
    assert fn(h=D + 4) == awq.AWQ_ERR_ALIGNMENT
    assert fn(h=A + 16) == awq.AWQ_ERR_INVALID_ARG           # h may be x, not a shifted x
    assert fn(h=B + 16) == awq.AWQ_ERR_INVALID_ARG
    assert fn(h=C) == awq.AWQ_ERR_INVALID_ARG
    assert fn(h=E) == awq.AWQ_ERR_INVALID_ARG                # h on y, or on x8
    assert fn(M=0) == awq.AWQ_OK


def test_rmsnorm_outputs():
    assert _norm(y=None) == awq.AWQ_ERR_INVALID_ARG
    assert _norm(y=A) == awq.AWQ_ERR_INVALID_ARG
    assert _norm(y=E + 2) == awq.AWQ_ERR_ALIGNMENT
    assert _norm8(x8=None) == awq.AWQ_ERR_INVALID_ARG
    assert _norm8(sx=None) == awq.AWQ_ERR_INVALID_ARG
    assert _norm8(sx=E + 16) == awq.AWQ_ERR_INVALID_ARG      # sx inside x8
    assert _norm8(h=F) == awq.AWQ_ERR_INVALID_ARG            # h on sx
    assert _norm8(sx=F + 4) == awq.AWQ_ERR_ALIGNMENT


def test_silu_refusals():
    def fp16(gu=A, y=B, M=4, F=256):
        return L.awq_silu_mul(gu, y, M, F, None)

    def fp8(gu=A, y=B, M=4, F=256, sx=C):
        return L.awq_silu_mul_fp8(gu, y, sx, M, F, None)

    for fn in (fp16, fp8):
        assert fn(M=-1) == awq.AWQ_ERR_SHAPE
        assert fn(F=0) == awq.AWQ_ERR_SHAPE
        assert fn(F=12) == awq.AWQ_ERR_SHAPE
        assert fn(F=1 << 23) == awq.AWQ_ERR_UNSUPPORTED
        assert fn(M=1 << 25) == awq.AWQ_ERR_UNSUPPORTED
        assert fn(M=1 << 24, F=1 << 20) == awq.AWQ_ERR_UNSUPPORTED
        assert fn(gu=None) == awq.AWQ_ERR_INVALID_ARG
        assert fn(y=None) == awq.AWQ_ERR_INVALID_ARG
        assert fn(y=A + 1024) == awq.AWQ_ERR_INVALID_ARG
        assert fn(gu=A + 2) == awq.AWQ_ERR_ALIGNMENT
        assert fn(M=0, gu=None, y=None) == awq.AWQ_OK
    assert fp8(sx=B) == awq.AWQ_ERR_INVALID_ARG
    assert fp8(sx=None) == awq.AWQ_ERR_INVALID_ARG


def _cache(**kw):
    v = dict(k=A, v=B, k_exp=C, v_exp=D, blocks=100, heads=8, block_tokens=64, head_dim=128)
    return awq._Kv8Cache(**{**v, **kw})


def _batch(**kw):
    v = dict(starts=E, lens=E + 4096, table=E + 8192, rows=3, seqs=2, table_width=10)
    return awq._Kv8Batch(**{**v, **kw})


WS_BYTES = 1 << 26


def _append(c=None, b=None, k=F, v=G, k_stride=1024, v_stride=1024, ws=H, ws_bytes=WS_BYTES):
    return L.awq_kv8_append(k, k_stride, v, v_stride, ctypes.byref(c or _cache()), ctypes.byref(b or _batch()), ws, ws_bytes,
                            None)


def _attend(c=None, b=None, q=F, q_stride=4096, q_heads=32, scale=0.1, y=G, ws=H, ws_bytes=WS_BYTES):
    return L.awq_kv8_attention(q, q_stride, q_heads, scale, ctypes.byref(c or _cache()), ctypes.byref(b or _batch()), y, ws,
                               ws_bytes, None)


@pytest.mark.parametrize("fn", [_append, _attend])
def test_kv8_shared_refusals(fn):
    S, U, I, P = awq.AWQ_ERR_SHAPE, awq.AWQ_ERR_UNSUPPORTED, awq.AWQ_ERR_INVALID_ARG, awq.AWQ_ERR_ALIGNMENT
    for kw, code in ((dict(blocks=0), S), (dict(blocks=-1), S), (dict(heads=0), S), (dict(heads=-8), S),
                     (dict(head_dim=96), U), (dict(head_dim=256), U), (dict(block_tokens=8), U), (dict(block_tokens=48), U),
                     (dict(block_tokens=256), U), (dict(blocks=1 << 31), U),
                     (dict(blocks=1 << 22), U),              # 2^31 rows of codes
                     (dict(k=None), I), (dict(v=None), I), (dict(k_exp=None), I), (dict(v_exp=None), I),
                     (dict(k=A + 8), P), (dict(v=B + 1), P),
                     (dict(v=A + 4096), I), (dict(k_exp=A), I), (dict(v_exp=C + 5), I)):
        assert fn(c=_cache(**kw)) == code, kw
    for kw, code in ((dict(rows=-1), S), (dict(seqs=-1), S), (dict(table_width=0), S), (dict(table_width=-1), S),
                     (dict(rows=(1 << 24) + 1), U), (dict(seqs=(1 << 20) + 1), U), (dict(table_width=1 << 23), U),
                     (dict(starts=None), I), (dict(lens=None), I), (dict(table=None), I),
                     (dict(starts=E + 2), P), (dict(table=E + 8193), P),
                     (dict(lens=C + 4), I), (dict(table=A), I)):
        assert fn(b=_batch(**kw)) == code, kw
    assert fn(ws=None) == I
    assert fn(ws=H + 4) == P
    assert fn(ws_bytes=256) == awq.AWQ_ERR_WORKSPACE
    assert fn(ws=A) == I                                     # the workspace on the cache
    assert fn(b=_batch(rows=0, starts=None, lens=None, table=None)) == awq.AWQ_OK
    assert fn(b=_batch(seqs=0, starts=None, lens=None, table=None), ws=None, ws_bytes=WS_BYTES) == awq.AWQ_OK


def test_kv8_append_refusals():
    assert _append(k=None) == awq.AWQ_ERR_INVALID_ARG
    assert _append(v=None) == awq.AWQ_ERR_INVALID_ARG
    assert _append(k=F + 8) == awq.AWQ_ERR_ALIGNMENT
    assert _append(k_stride=1016) == awq.AWQ_ERR_SHAPE       # shorter than a row
    assert _append(v_stride=1028) == awq.AWQ_ERR_SHAPE       # not a multiple of 8
    assert _append(k_stride=-1024) == awq.AWQ_ERR_SHAPE
    assert _append(k=A + 64) == awq.AWQ_ERR_INVALID_ARG      # k inside the cache
    assert _append(v=C) == awq.AWQ_ERR_INVALID_ARG


def test_kv8_attention_refusals():
    assert _attend(q_heads=0) == awq.AWQ_ERR_SHAPE
    assert _attend(q_heads=36) == awq.AWQ_ERR_SHAPE          # not a multiple of the kv heads
    assert _attend(q_heads=8192, q_stride=8192 * 128) == awq.AWQ_ERR_UNSUPPORTED
    assert _attend(q=None) == awq.AWQ_ERR_INVALID_ARG
    assert _attend(y=None) == awq.AWQ_ERR_INVALID_ARG
    assert _attend(y=F) == awq.AWQ_ERR_INVALID_ARG           # y on q
    assert _attend(y=B + 1024) == awq.AWQ_ERR_INVALID_ARG    # y on the cache
    assert _attend(y=H) == awq.AWQ_ERR_INVALID_ARG           # y on the workspace
    assert _attend(y=E) == awq.AWQ_ERR_INVALID_ARG           # y on the batch's lists
    assert _attend(q=F + 8) == awq.AWQ_ERR_ALIGNMENT
    assert _attend(q_stride=4088) == awq.AWQ_ERR_SHAPE
    assert _attend(q_stride=4100) == awq.AWQ_ERR_SHAPE
    for s in (float("nan"), float("inf")):
        assert _attend(scale=s) == awq.AWQ_ERR_INVALID_ARG


def test_kv8_null_structs():
    c, b = _cache(), _batch()
    assert L.awq_kv8_append(F, 1024, G, 1024, None, ctypes.byref(b), H, WS_BYTES, None) == awq.AWQ_ERR_INVALID_ARG
    assert L.awq_kv8_attention(F, 4096, 32, 0.1, ctypes.byref(c), None, G, H, WS_BYTES, None) == awq.AWQ_ERR_INVALID_ARG


def test_kv8_workspace_bytes():
    assert awq.awq_kv8_workspace_bytes(1, 1, 32, 8, 128) > 256
    assert awq.awq_kv8_workspace_bytes(1, 1, 32, 8, 64) < awq.awq_kv8_workspace_bytes(1, 1, 32, 8, 128) < WS_BYTES
    for bad in ((-1, 1, 32, 8, 128), (1, -1, 32, 8, 128), (1, 1, 0, 8, 128), (1, 1, 30, 8, 128), (1, 1, 32, 8, 80),
                (1, 1, 32, 0, 128), (1 << 25, 1, 32, 8, 128), (1 << 20, 1, 4096, 8, 128)):
        assert awq.awq_kv8_workspace_bytes(*bad) == 0, bad


def test_binding_rejects_what_is_not_on_a_gpu():
    x = torch.zeros(2, 128, dtype=torch.float16)
    with pytest.raises(ValueError):
        awq.awq_rmsnorm(x, x[0], 1e-5)
    with pytest.raises(ValueError):
        awq.awq_silu_mul(x)
    with pytest.raises(ValueError):
        awq.awq_silu_mul(x[:, :127])
    cache = awq.Kv8Cache(torch.zeros(1, 2, 16, 64, dtype=torch.uint8), torch.zeros(1, 2, 16, 64, dtype=torch.uint8),
                         torch.zeros(1, 2, dtype=torch.int8), torch.zeros(1, 2, dtype=torch.int8))
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        awq.awq_kv8_attention(torch.zeros(1, 2, 64, dtype=torch.float16), cache, i, i[:1], i[:1].view(1, 1),
                              torch.zeros(256, dtype=torch.uint8))


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch with fake pointers on a GPU")
def test_valid_arguments_without_a_device_stop_at_the_device_check():
    assert _norm() == awq.AWQ_ERR_UNSUPPORTED
    assert _norm(h=A) == awq.AWQ_ERR_UNSUPPORTED             # in place
    assert _norm(h=B) == awq.AWQ_ERR_UNSUPPORTED
    assert _norm(residual=None, h=None) == awq.AWQ_ERR_UNSUPPORTED
    assert _norm8() == awq.AWQ_ERR_UNSUPPORTED
    assert L.awq_silu_mul(A, B, 4, 256, None) == awq.AWQ_ERR_UNSUPPORTED
    assert L.awq_silu_mul_fp8(A, B, C, 4, 256, None) == awq.AWQ_ERR_UNSUPPORTED
    assert _append() == awq.AWQ_ERR_UNSUPPORTED
    assert _append(k=F, v=F + 2048, k_stride=6144, v_stride=6144) == awq.AWQ_ERR_UNSUPPORTED   # ranges of one matrix
    assert _attend() == awq.AWQ_ERR_UNSUPPORTED


def test_kv8_attention_refuses_scales_beyond_its_scores():
    # above 2^32 a row whose scores are all large and negative would count as one without keys
    for s in (2.0 ** 32 * 1.001, -(2.0 ** 33), 1e30, -1e38):
        assert _attend(scale=s) == awq.AWQ_ERR_UNSUPPORTED
    for s in (2.0 ** 32, -(2.0 ** 32), 0.0):
        assert _attend(scale=s, y=None) == awq.AWQ_ERR_INVALID_ARG       # gets past the scale
