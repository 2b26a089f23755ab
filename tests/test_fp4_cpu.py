"""Host-side refusals of attention over a 4-bit cache (CPU only: fake
addresses, every call is answered before anything is enqueued)."""
import ctypes

import pytest
import torch

P = 0x10000


@pytest.fixture(scope="module")
def capi():
    from top_sparse_attention_qsa_b200 import build
    build.build()
    from top_sparse_attention_qsa_b200 import _capi
    return _capi


def _shape(capi, **kw):
    base = dict(num_tokens=4, num_q_heads=12, num_kv_heads=1, head_dim=256, topk=300, num_slots=64,
                q_stride_tok=12 * 256, q_stride_head=256, kv_stride_slot=288, kv_stride_head=288, idx_stride_tok=300,
                idx_stride_head=300, o_stride_tok=12 * 256, o_stride_head=256, lse_stride_tok=12)
    base.update(kw)
    return capi.Shape(**base)


def _prefill(capi, s, bs=1, q=P, kc=P, kb=P, vc=P, vb=P, ss=288, sh=288, idx=P, out=P):
    return capi.library().qsa_sparse_prefill_fp4_fwd(ctypes.byref(s) if s is not None else None, bs, None, q, kc, kb, vc,
                                                     vb, ss, sh, idx, None, 0.0, 1.0, 1.0, out, None, None, None)


def _decode(capi, s, ws=P, n=1 << 30, splits=2):
    return capi.library().qsa_sparse_decode_fp4_fwd(ctypes.byref(s), P, P, P, P, P, 288, 288, P, None, 0.0, 1.0, 1.0, P,
                                                    None, None, splits, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=128), 3),
    (dict(num_q_heads=17), 3),
    (dict(num_slots=1 << 31), 3),
    (dict(topk=2 ** 31 - 100), 3),
    (dict(kv_stride_slot=1 << 31), 3),
    (dict(num_tokens=-1), 2),
    (dict(kv_stride_slot=0), 2),
    (dict(kv_stride_slot=-288), 2),
    (dict(q_stride_head=260), 4),
    (dict(kv_stride_slot=296), 4),
    (dict(kv_stride_head=136), 4),
])
def test_shape_refusals(capi, kw, code):
    assert _prefill(capi, _shape(capi, **kw)) == code
    assert _decode(capi, _shape(capi, **kw)) == code


def test_null_and_alignment(capi):
    s = _shape(capi)
    assert _prefill(capi, None) == 1
    for name in ("q", "kc", "kb", "vc", "vb", "idx", "out"):
        assert _prefill(capi, s, **{name: None}) == 1, name
        assert _prefill(capi, s, **{name: P + (2 if name == "idx" else 8)}) == 4, name
    assert _prefill(capi, s, ss=0) == 2
    assert _prefill(capi, s, sh=-16) == 2
    assert _prefill(capi, s, ss=296) == 4
    assert _prefill(capi, s, ss=1 << 31) == 3
    assert _prefill(capi, s, bs=3) == 3
    assert _prefill(capi, _shape(capi, topk=1 << 28), bs=16) == 3
    assert _prefill(capi, _shape(capi, num_tokens=0), q=None, out=None) == 0


def test_decode_workspace(capi):
    s = _shape(capi)
    assert _decode(capi, s, ws=None) == 1
    assert _decode(capi, s, n=64) == 2
    assert _decode(capi, s, ws=P + 16) == 4


def test_binding_refusals(capi):
    q = torch.zeros(2, 3, 256, dtype=torch.bfloat16)
    idx = torch.zeros(2, 1, 4, dtype=torch.int32)
    cache = capi.fp4_cache(8, 1, device="cpu")
    with pytest.raises(ValueError):                      # host tensors
        capi.sparse_prefill_fp4_fwd(q, cache, idx, 1.0, 1.0)
    with pytest.raises(TypeError):
        capi.sparse_decode_fp4_fwd(q.float(), cache, idx, 1.0, 1.0)
