"""What a decode over a 4-bit cache does in all its forms: one chunk, chunks
merged in a cluster, chunks merged from a workspace.  Tolerances are those of
test_gpu_fp4.py."""
import ctypes

import numpy as np
import pytest
import torch

import cache_ref as R
from test_gpu_fp4 import case, compare, reference
from top_sparse_attention_qsa_b200 import workloads as W

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = "cuda"


@pytest.fixture(scope="module")
def C():
    from top_sparse_attention_qsa_b200 import _capi
    return _capi


def test_named_workspace_is_checked_with_or_without_clusters(C):
    """A workspace that is named for a given chunk count is checked against that
    count on every device, whether or not its chunks run as clusters there."""
    T, ctx, K, heads = 4, 400, 300, (12, 1)
    q, cache, ks, vs, g = case(C, T, T * ctx, heads, seed=92)
    idx = W.random_lists(T, 1, K, ctx, g, DEV) + (torch.arange(T, dtype=torch.int32, device=DEV) * ctx).view(T, 1, 1)
    ref = reference(q, cache, ks, vs, idx)
    call = lambda **kw: C.sparse_decode_fp4_fwd(q, cache, idx, ks, vs, num_splits=2, **kw)  # noqa: E731
    need = C.decode_fp4_workspace_bytes(q, cache, idx, 2)
    assert need == T * 12 * 2 * (256 + 1) * 4
    room = torch.full((need + 256,), 0xff, dtype=torch.uint8, device=DEV)
    for ws, code in ((room[:64], 2), (room[:need - 4], 2), (room[16:16 + need], 4)):
        with pytest.raises(C.QSAError) as e:
            call(workspace=ws)
        assert e.value.code == code
    # NULL with a number of bytes names one too; NULL with none is a call without a workspace
    shape = C.make_shape(q, cache.buffer, idx, q)
    base, out = cache.buffer.data_ptr(), torch.empty_like(q)
    raw = lambda ws, n: C.library().qsa_sparse_decode_fp4_fwd(  # noqa: E731
        ctypes.byref(shape), q.data_ptr(), base, base + 256, base + 128, base + 272, 288, 288, idx.data_ptr(), None, 0.0,
        ks, vs, out.data_ptr(), None, None, 2, ws, n, torch.cuda.current_stream().cuda_stream)
    assert raw(None, 1 << 30) == 1
    assert raw(None, 0) in (0, 1)                        # (1: a device whose clusters do not fit)
    torch.cuda.synchronize()
    for kw in ({}, {"workspace": room}, {"workspace": room[:need]}):
        out, lse = call(**kw)
        torch.cuda.synchronize()
        assert compare(out, lse, ref, str(list(kw))) == 0


FORMS = {"one chunk": (6, 1), "cluster": (6, 0), "workspace": (40, 3)}


@pytest.mark.parametrize("heads", [(24, 2), (16, 2)])
@pytest.mark.parametrize("form", FORMS)
def test_nan_in_every_decode_form(C, form, heads):
    """A NaN in a query head, a K or a V block scale gives NaN where the formula
    does and nowhere else, with empty chunks and empty lists beside it."""
    T, splits = FORMS[form]
    ctx, K = 700, 650
    G = heads[0] // 2
    q, cache, ks, vs, g = case(C, T, T * ctx, heads, seed=91)
    idx = W.random_lists(T, 2, K, ctx, g, DEV) + (torch.arange(T, dtype=torch.int32, device=DEV) * ctx).view(T, 1, 1)
    nv = torch.full((T, 2), K, dtype=torch.int32, device=DEV)
    nv[1], nv[2], nv[3, 0] = 0, 200, 1                   # an empty list, a chunk with keys beside empty ones, one key
    if form != "one chunk":
        assert (C.decode_fp4_workspace_bytes(q, cache, idx, splits) > 0) == (form == "workspace")
    ref = reference(q, cache, ks, vs, idx, nv)
    hit = np.zeros((T, heads[0]), dtype=bool)

    def run(q, buf):
        out, lse = C.sparse_decode_fp4_fwd(q, C.Fp4Cache(buf), idx, ks, vs, n_valid=nv, num_splits=splits)
        torch.cuda.synchronize()
        return out, lse

    def clean_outside(out, lse):
        """Rows that were not hit are the clean ones (the hit ones replaced by the reference)."""
        h = torch.from_numpy(hit).to(DEV)
        out, lse = out.clone(), lse.clone()
        out[h] = torch.from_numpy(ref[0]).to(DEV)[h].to(torch.bfloat16)
        lse[h] = torch.from_numpy(ref[1]).to(DEV)[h].float()
        assert compare(out, lse, ref, form) == heads[0]

    # query elements: a long list, one with empty chunks, one of a single key; a head without a key stays empty
    bad = q.clone()
    for t, h in ((0, 3), (2, 5), (3, 0), (5, G)):
        bad[t, h, 9] = float("nan")
        hit[t, h] = True
    bad[1, 2, 9] = float("nan")
    out, lse = run(bad, cache.buffer)
    o, l = R.f64(out), R.f64(lse)
    assert np.isnan(o[hit]).all() and np.isnan(l[hit]).all()
    clean_outside(out, lse)

    # one K block scale: every head of the KV head of the tokens that name the row
    for t, j in ((0, 600), (0, 3), (2, 190), (3, 0)):
        hit[:] = False
        hit[t, :G] = True
        buf = cache.buffer.clone()
        buf[int(idx[t, 0, j]), 0, 256 + 5] = 0x7f
        out, lse = run(q, buf)
        o, l = R.f64(out), R.f64(lse)
        assert np.isnan(o[hit]).all() and np.isnan(l[hit]).all(), (t, j)
        clean_outside(out, lse)

    # one V block scale: its 16 dims; the lse is not touched
    hit[:] = False
    hit[2, G:] = True
    buf = cache.buffer.clone()
    buf[int(idx[2, 1, 150]), 1, 272 + 3] = 0x7f
    out, lse = run(q, buf)
    o = R.f64(out)
    assert np.isnan(o[hit][:, 48:64]).all() and np.isfinite(np.delete(o[hit], np.s_[48:64], -1)).all()
    assert np.all(np.abs(R.f64(lse)[hit] - ref[1][hit]) <= ref[3][hit])
    clean_outside(out, lse)


def test_rows_of_another_width_are_refused(C):
    """A buffer put into an Fp4Cache past its constructor is checked by the calls."""
    q, cache, ks, vs, g = case(C, 2, 64, (12, 1), seed=93)
    idx = W.random_lists(2, 1, 8, 64, g, DEV)
    k = torch.zeros((2, 1, 256), dtype=torch.bfloat16, device=DEV)
    pos = torch.arange(2, dtype=torch.int32, device=DEV)
    before = cache.buffer.clone()
    whole = cache.buffer
    cache.buffer = whole[..., :256]
    for call in (lambda: C.sparse_prefill_fp4_fwd(q, cache, idx, ks, vs),
                 lambda: C.sparse_decode_fp4_fwd(q, cache, idx, ks, vs),
                 lambda: C.kv_append_fp4(k, k, pos, pos, None, cache, ks, vs)):
        with pytest.raises(ValueError, match="288"):
            call()
    torch.cuda.synchronize()
    assert torch.equal(whole, before)
