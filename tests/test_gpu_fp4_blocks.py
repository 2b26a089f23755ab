"""Microblock lists over a 4-bit cache in every form of the kernels: wide and
narrow, 8 (12), 4, 2 warps to a unit and one.  Tolerances are those of
test_gpu_fp4.py."""
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


@pytest.mark.parametrize("heads", [(12, 1), (6, 1), (16, 2)])
@pytest.mark.parametrize("units", [100, 250, 500, 900])
@pytest.mark.parametrize("bs", [1, 4, 16])
def test_block_forms(C, heads, units, bs):
    """Lists of about 600 keys; a cache that ends inside a block, ragged counts,
    holes, blocks past the end, last slots inside a block, tokens that see nothing."""
    S, Hkv = 1203, heads[1]
    T, K, nb = units // Hkv, 600 // bs, (S + bs - 1) // bs
    q, cache, ks, vs, g = case(C, T, S, heads, seed=units + bs)
    idx = W.random_lists(T, Hkv, K, nb, g, DEV)
    idx[::7, :, 0] = nb - 1                              # the block that the cache's end cuts
    idx[::5, :, 2] = -1
    idx[4, :, 1] = nb
    nv = torch.randint(0, K + 1, (T, Hkv), generator=g, device=DEV, dtype=torch.int32)
    nv[::3] = K
    nv[1] = 0
    last = torch.randint(S // 3, S, (T,), generator=g, device=DEV, dtype=torch.int32)
    last[::4] = S - 1
    last[2] = -1
    nv[4] = K
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = C.sparse_prefill_fp4_fwd(q, cache, idx, ks, vs, n_valid=nv, block_size=bs, last_slot=last, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == C.STATUS_OOB_SLOT
    t = sorted({0, 1, 2, 3, 4, 7, T - 2, T - 1, *range(0, T, 37)})
    ti = torch.tensor(t)
    ref = reference(q, cache, ks, vs, idx, nv, tokens=t, block_size=bs, last_slot=last)
    assert compare(out[ti], lse[ti], ref, f"{heads} {units} {bs}") >= 2 * heads[0]
