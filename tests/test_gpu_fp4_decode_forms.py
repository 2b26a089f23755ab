"""What a decode over a 4-bit cache does in all its forms: one chunk, chunks
merged in a cluster, chunks merged from a workspace.  Tolerances are those of
test_gpu_fp4.py."""
import ctypes

import pytest
import torch

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
