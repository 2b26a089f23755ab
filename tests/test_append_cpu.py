"""Host-side refusals of the cache appends (CPU only: fake addresses, every
call is answered before anything is enqueued)."""
import ctypes

import numpy as np
import pytest
import torch

import cache_ref as R

P = 0x10000


@pytest.fixture(scope="module")
def capi():
    from top_sparse_attention_qsa_b200 import build
    build.build()
    from top_sparse_attention_qsa_b200 import _capi
    return _capi


def _shape(capi, **kw):
    base = dict(num_tokens=4, num_q_heads=12, num_kv_heads=2, head_dim=256, rotary_dim=64, interleaved=0, reserved=0,
                num_slots=64, num_positions=128, q_stride_tok=12 * 256, q_stride_head=256, qo_stride_tok=12 * 256,
                qo_stride_head=256, k_stride_tok=512, k_stride_head=256, v_stride_tok=512, v_stride_head=256,
                table_stride=64, kv_stride_slot=576, kv_stride_head=288, bscale_stride_slot=576,
                bscale_stride_head=288)
    base.update(kw)
    return capi.AppendShape(**base)


def _fp4(capi, s, q=P, qo=P, k=P, v=P, tab=P, pos=P, slots=P, ks=1.0, vs=1.0, kc=P, kb=P, vc=P, vb=P, seen=None):
    return capi.library().qsa_kv_append_fp4(ctypes.byref(s) if s is not None else None, q, qo, k, v, tab, pos, slots,
                                            ks, vs, kc, kb, vc, vb, seen, None, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=128), 3),
    (dict(rotary_dim=24), 3),
    (dict(rotary_dim=272), 3),
    (dict(interleaved=2), 3),
    (dict(reserved=1), 3),
    (dict(num_tokens=1 << 28), 3),                       # rows no 32-bit count holds
    (dict(num_slots=(1 << 31) + 1), 3),
    (dict(num_tokens=-1), 2),
    (dict(num_kv_heads=0), 2),
    (dict(num_q_heads=-1), 2),
    (dict(k_stride_tok=-512), 2),
    (dict(table_stride=60), 2),
    (dict(kv_stride_slot=0), 2),                         # rows that are written overlap
    (dict(kv_stride_slot=288), 2),                       # slots overlap the next slot's heads
    (dict(kv_stride_head=112), 2),
    (dict(bscale_stride_head=0), 2),
    (dict(q_stride_tok=6 * 256, qo_stride_tok=6 * 256), 2),
    (dict(q_stride_tok=24 * 256), 2),                    # in place with other strides
    (dict(k_stride_head=260), 4),
    (dict(kv_stride_slot=584), 4),
    (dict(bscale_stride_slot=584), 4),
    (dict(table_stride=66), 4),
])
def test_shape_refusals(capi, kw, code):
    assert _fp4(capi, _shape(capi, **kw)) == code


def test_null_alignment_and_scales(capi):
    s = _shape(capi)
    assert _fp4(capi, None) == 1
    for name in ("q", "qo", "k", "v", "tab", "pos", "slots", "kc", "kb", "vc", "vb"):
        assert _fp4(capi, s, **{name: None}) == 1, name
        odd = P + (2 if name in ("pos", "slots") else 8)
        assert _fp4(capi, s, **{name: odd}) == 4, name
    assert _fp4(capi, s, seen=P + 2) == 4
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e-38, 1e38):
        assert _fp4(capi, s, ks=bad) == 3
        assert _fp4(capi, s, vs=bad) == 3
    # no tokens: nothing is read; head-major caches do not overlap
    assert _fp4(capi, _shape(capi, num_tokens=0), q=None, k=None, slots=None) == 0
    hm = _shape(capi, kv_stride_slot=144, kv_stride_head=64 * 144, bscale_stride_slot=144,
                bscale_stride_head=64 * 144)
    assert _fp4(capi, hm, vb=P + 8) == 4                 # past the overlap checks
    hm = _shape(capi, kv_stride_slot=144, kv_stride_head=63 * 144, bscale_stride_slot=144,
                bscale_stride_head=64 * 144)
    assert _fp4(capi, hm) == 2


def test_bf16_and_fp8_entries(capi):
    lib = capi.library()
    s = _shape(capi, kv_stride_slot=512, kv_stride_head=256)
    bf = lambda s, vc=P: lib.qsa_kv_append(ctypes.byref(s), P, P, P, P, P, P, P, P, vc, None, None)  # noqa: E731
    assert bf(s, None) == 1
    assert bf(_shape(capi, kv_stride_slot=520, kv_stride_head=260)) == 4
    assert bf(_shape(capi, kv_stride_slot=256, kv_stride_head=256)) == 2
    f8 = lambda s, ks=1.0: lib.qsa_kv_append_fp8(ctypes.byref(s), P, P, P, P, P, P, P, ks, 1.0, P, P, None, None,  # noqa: E731
                                                 None, None)
    assert f8(s, 0.0) == 3
    assert f8(_shape(capi, kv_stride_slot=528, kv_stride_head=264)) == 4


def test_binding_refusals(capi):
    k = torch.zeros(2, 1, 256, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):                      # host tensors
        capi.kv_append(k, k, i, i, None, k, k)
    with pytest.raises(TypeError):
        capi.kv_append(k.float(), k, i, i, None, k, k)
    with pytest.raises(TypeError):
        capi.Fp4Cache(torch.zeros(4, 1, 288))
    with pytest.raises(ValueError):
        capi.Fp4Cache(torch.zeros(4, 1, 256, dtype=torch.uint8))
    c = capi.fp4_cache(5, 2, device="cpu")
    assert c.k_codes.shape == c.v_codes.shape == (5, 2, 128)
    assert c.k_bscale.shape == c.v_bscale.shape == (5, 2, 16)
    assert c.v_codes.data_ptr() - c.k_codes.data_ptr() == 128
    assert c.v_bscale.data_ptr() - c.k_codes.data_ptr() == 272


def test_rope_table(capi):
    t = capi.rope_table(70000, 64, base=1e6, device="cpu")
    assert t.shape == (70000, 64) and t.dtype == torch.float32
    p, i = 69999, 3
    a = np.float64(p) * np.float64(1e6) ** (-2 * i / 64)
    # one rounding to FP32 of values at most 1, and the FP64 angle's own error
    assert abs(float(t[p, i]) - np.cos(a)) < 2.0 ** -24
    assert abs(float(t[p, 32 + i]) - np.sin(a)) < 2.0 ** -24


def test_reference_formats():
    """The test's own E4M3 and E2M1 roundings against torch's E4M3 and a hand count."""
    x = np.linspace(-500, 500, 4001)
    x = np.concatenate([x, x / 4096, np.exp2(np.arange(-12, 9)) * 1.0625])
    t = torch.from_numpy(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.e4m3(x.astype(np.float32).astype(np.float64)), t)
    y = np.zeros((1, 256))
    y[0, :10] = [6, 5, 5.01, 2.5, 0.25, 0.26, -0.75, 1.25, -3.5, 1.75]
    code, e, val = R.fp4_encode(y, 1.0)
    assert e[0, 0] == 1.0 and e[0, 1] == 0.0
    assert list(code[0, :10]) == [7, 6, 7, 4, 0, 1, 10, 2, 14, 4]
    assert list(val[0, :10]) == [6, 4, 6, 2, 0, 0.5, -1, 1, -4, 2]
