"""Attention over a 4-bit cache against FP64 attention over the decoded rows.

Tolerance.  Of a head's scores, mass = max_j scale * sum_d |q_d k_jd| bounds
every partial sum.  The 256 products are exact in FP32 and are added in 16
steps of 16 (each at most two roundings or truncations to 24 bits, 2^-23):
a score is off by at most eps = 2^-18 mass, and a probability by a factor of
1 +- 2 eps.  Probabilities are rounded to FP16, 2^-11 relative, or, where they
underflow, by half of FP16's smallest step after the scaling by 2^7: 2^-32 of
the largest.  exp2 and the FP32 sums of up to 2^12 terms add less than 2^-11.
The output is rounded to BF16, 2^-8.  With A = sum_j p_j |v_j| / l and B =
sum_j |v_j| over the list,
  |out - ref| <= 2^-8 |ref| + (2^-10 + 2 eps) A + 2^-32 B
  |lse - ref| <= eps + 2^-18 (1 + |ref|)
"""
import numpy as np
import pytest
import torch

import cache_ref as R
from parity import host
from top_sparse_attention_qsa_b200 import workloads as W

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = "cuda"


@pytest.fixture(scope="module")
def C():
    from top_sparse_attention_qsa_b200 import _capi
    return _capi


def case(C, T, S, heads, seed, spread=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randn((T, heads[0], 256), generator=g, device=DEV).to(torch.bfloat16)
    buf, ks, vs = R.fp4_buffer(S, heads[1], seed + 1, DEV, spread)
    return q, C.Fp4Cache(buf), ks, vs, g


def reference(q, cache, ks, vs, idx, nv=None, **kw):
    k, v = R.fp4_rows(cache.buffer)
    return reference_rows(q, k * np.float64(np.float32(ks)), v * np.float64(np.float32(vs)), idx, nv, **kw)


def reference_rows(q, k, v, idx, nv=None, **kw):
    """(out, lse, bound of out, bound of lse) of attention over float64 rows."""
    out, lse = R.attention(q, k, v, idx, nv, **kw)
    A, _ = R.attention(q, k, np.abs(v), idx, nv, **kw)
    flat, _ = R.attention(q * 0, k, np.abs(v), idx, nv, **kw)       # mean |v| of the list
    B = flat * idx.shape[2] * kw.get("block_size", 1)
    scale = kw.get("scale", 1 / 16)
    tokens = list(kw.get("tokens", range(q.shape[0])))
    G = q.shape[1] // k.shape[1]
    qa = np.abs(R.f64(q))[tokens]
    mass = np.stack([(qa[:, h] @ np.abs(k[:, h // G]).T).max(1) for h in range(q.shape[1])], 1) * scale
    eps = 2.0 ** -18 * mass
    with np.errstate(invalid="ignore"):
        return (out, lse, 2.0 ** -8 * np.abs(out) + (2.0 ** -10 + 2 * eps[..., None]) * A + 2.0 ** -32 * B + 1e-300,
                eps + 2.0 ** -18 * (1 + np.abs(lse)))


def compare(out, lse, ref, label=""):
    ro, rl, bo, bl = ref
    o, l = R.f64(out), R.f64(lse)
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(l), empty), f"{label}: empty rows"
    assert np.all(host(out).contiguous().view(torch.int16).numpy()[empty] == 0), f"{label}: empty rows not +0"
    assert np.isfinite(o).all(), f"{label}: non-finite output"
    d = np.abs(o - ro)[~empty]
    worst = float((d / bo[~empty]).max())
    assert worst <= 1, f"{label}: out off by {d.max():.3e}, {worst:.2f} of the bound"
    d = np.abs(l[~empty] - rl[~empty])
    worst = float((d / bl[~empty]).max())
    assert worst <= 1, f"{label}: lse off by {d.max():.3e}, {worst:.2f} of the bound"
    return int(empty.sum())


@pytest.mark.parametrize("heads", [(3, 1), (6, 1), (12, 1), (16, 2), (24, 2), (16, 1), (1, 1), (5, 5)])
def test_head_shapes_ragged(C, heads):
    # K = 700: five 128-key tiles and a ragged one; ragged n_valid
    T, S = 17, 1500
    q, cache, ks, vs, g = case(C, T, S, heads, seed=heads[0] * 7 + heads[1], spread=2.0)
    idx = W.random_lists(T, heads[1], 700, S, g, DEV)
    nv = torch.randint(0, 701, (T, heads[1]), generator=g, device=DEV, dtype=torch.int32)
    nv[0] = 700
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = C.sparse_prefill_fp4_fwd(q, cache, idx, ks, vs, n_valid=nv, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    compare(out, lse, reference(q, cache, ks, vs, idx, nv), f"{heads}")


@pytest.mark.parametrize("K", [1, 2, 127, 128, 129, 256, 385])
def test_list_lengths(C, K):
    T, S, heads = 5, 400, (12, 1)
    q, cache, ks, vs, g = case(C, T, S, heads, seed=K)
    idx = W.random_lists(T, 1, K, S, g, DEV)
    out, lse = C.sparse_prefill_fp4_fwd(q, cache, idx, ks, vs, scale=0.11)
    torch.cuda.synchronize()
    compare(out, lse, reference(q, cache, ks, vs, idx, scale=np.float64(np.float32(0.11))), f"K={K}")


def test_masks_empty_rows_and_out_of_range(C):
    T, S, heads = 12, 900, (16, 2)
    q, cache, ks, vs, g = case(C, T, S, heads, seed=5)
    idx = W.random_lists(T, 2, 300, S, g, DEV)
    idx[3] = -1                                          # empty rows
    idx[5, 1, 17] = S                                    # out of range: masked and reported
    idx[6, 0, 3] = 2 ** 31 - 1
    idx[7, 0, ::3] = -1                                  # interior holes
    idx[8, 0, :128] = -1                                 # an empty first tile
    idx[9, 1, 128:] = -(2 ** 31)
    idx[10, 0, 5:250] = idx[10, 0, 4]                    # one slot many times
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = C.sparse_prefill_fp4_fwd(q, cache, idx, ks, vs, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == C.STATUS_OOB_SLOT
    assert compare(out, lse, reference(q, cache, ks, vs, idx), "masks") == 16


def test_zero_keys_and_no_cache(C):
    T, heads = 4, (6, 1)
    q, cache, ks, vs, g = case(C, T, 8, heads, seed=6)
    idx = torch.zeros((T, 1, 0), dtype=torch.int32, device=DEV)
    out, lse = C.sparse_prefill_fp4_fwd(q, cache, idx, ks, vs, out=torch.full_like(q, 3.0))
    torch.cuda.synchronize()
    assert bool((out.view(torch.int16) == 0).all()) and bool((lse == -float("inf")).all())
    with pytest.raises(C.QSAError):                      # lists over a cache without a row: no base address
        C.sparse_prefill_fp4_fwd(q, C.Fp4Cache(cache.buffer[:0]), idx.new_zeros((T, 1, 5)), ks, vs)
    nv = torch.tensor([[0], [-3], [1], [0]], dtype=torch.int32, device=DEV)
    idx = torch.arange(5, dtype=torch.int32, device=DEV).repeat(T, 1, 1)
    out, lse = C.sparse_prefill_fp4_fwd(q, cache, idx, ks, vs, n_valid=nv)
    torch.cuda.synchronize()
    compare(out, lse, reference(q, cache, ks, vs, idx, nv), "n_valid")


def test_runs_of_empty_units(C):
    """Units per CTA alternating full, empty (runs of three), short and one-key
    lists, so that every two-buffer hand-off wraps its phases on empty units."""
    nsm = torch.cuda.get_device_properties(0).multi_processor_count
    pattern = [256, 0, 0, 0, 200, 0, 1, 256, 0, 130]
    T = nsm * len(pattern)
    q, cache, ks, vs, g = case(C, T, 1024, (16, 1), seed=23)
    idx = W.random_lists(T, 1, 256, 1024, g, DEV)
    nv = torch.tensor([pattern[t // nsm] for t in range(T)], dtype=torch.int32, device=DEV).reshape(T, 1)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = C.sparse_prefill_fp4_fwd(q, cache, idx, ks, vs, n_valid=nv, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    t = np.arange(0, T, 7)
    ref = reference(q, cache, ks, vs, idx, nv, tokens=list(t))
    compare(out[torch.from_numpy(t)], lse[torch.from_numpy(t)], ref, "empty units")


@pytest.mark.parametrize("heads", [(12, 1), (6, 1)])
@pytest.mark.parametrize("T", [100, 250, 500, 1400])
def test_warps_per_unit(C, heads, T):
    """Numbers of units for which a unit is worked by 8 (12), 4, 2 warps and by one."""
    S, K = 900, 600
    q, cache, ks, vs, g = case(C, T, S, heads, seed=T + heads[0])
    idx = W.random_lists(T, 1, K, S, g, DEV)
    nv = torch.randint(0, K + 1, (T, 1), generator=g, device=DEV, dtype=torch.int32)
    nv[::5] = K
    nv[3] = 0
    out, lse = C.sparse_prefill_fp4_fwd(q, cache, idx, ks, vs, n_valid=nv)
    torch.cuda.synchronize()
    t = sorted({0, 1, 2, 3, T - 2, T - 1, *range(0, T, 29)})
    ti = torch.tensor(t)
    assert compare(out[ti], lse[ti], reference(q, cache, ks, vs, idx, nv, tokens=t), f"T={T}") >= heads[0]


@pytest.mark.parametrize("heads", [(12, 1), (6, 1)])
@pytest.mark.parametrize("T,K", [(1200, 200), (1900, 200), (500, 30), (140, 40)])
def test_warps_per_short_unit(C, heads, T, K):
    """Short lists: one warp to a unit in one round and in two, and several warps with a group or two between them."""
    S = 500
    q, cache, ks, vs, g = case(C, T, S, heads, seed=T + K)
    idx = W.random_lists(T, 1, K, S, g, DEV)
    nv = torch.randint(0, K + 1, (T, 1), generator=g, device=DEV, dtype=torch.int32)
    nv[::5] = K
    nv[3] = 0
    out, lse = C.sparse_prefill_fp4_fwd(q, cache, idx, ks, vs, n_valid=nv)
    torch.cuda.synchronize()
    t = sorted({0, 1, 2, 3, T - 2, T - 1, *range(0, T, 29)})
    ti = torch.tensor(t)
    assert compare(out[ti], lse[ti], reference(q, cache, ks, vs, idx, nv, tokens=t), f"T={T}") >= heads[0]


def test_two_streams_at_once(C):
    """Appends and decodes of two batches on two streams, as when each runs alone."""
    runs = []
    for seed in (81, 82):
        q, cache, ks, vs, g = case(C, 9, 4000, (24, 2), seed)
        k, v = (torch.randn((9, 2, 256), generator=g, device=DEV).to(torch.bfloat16) for _ in "kv")
        pos = torch.randint(0, 4000, (9,), generator=g, device=DEV, dtype=torch.int32)
        slots = torch.randperm(4000, generator=g, device=DEV)[:9].to(torch.int32)
        idx = W.random_lists(9, 2, 1500, 4000, g, DEV)
        idx[:, :, 0] = slots.view(9, 1)
        runs.append((q, cache, ks, vs, k, v, pos, slots, idx))
    table = C.rope_table(4000, 64, device=DEV)

    def step(r, cache):
        q, _, ks, vs, k, v, pos, slots, idx = r
        qr, _, _ = C.kv_append_fp4(k, v, pos, slots, table, cache, ks, vs, q=q)
        return C.sparse_decode_fp4_fwd(qr, cache, idx, ks, vs)

    alone = [step(r, C.Fp4Cache(r[1].buffer.clone())) for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(5):
        caches = [C.Fp4Cache(r[1].buffer.clone()) for r in runs]
        torch.cuda.synchronize()
        outs = []
        for r, c, s in zip(runs, caches, streams):
            with torch.cuda.stream(s):
                outs.append(step(r, c))
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(outs, alone):
            assert torch.equal(o, wo) and torch.equal(l, wl)


@pytest.mark.parametrize("bs", [1, 2, 4, 16])
def test_block_lists_with_tail(C, bs):
    T, S = 9, 1203
    q, cache, ks, vs, g = case(C, T, S, (24, 2), seed=11 + bs)
    nb = (S + bs - 1) // bs
    K = min(nb, 520 // bs)
    idx = W.random_lists(T, 2, K, nb, g, DEV)
    nv = torch.randint(0, K + 1, (T, 2), generator=g, device=DEV, dtype=torch.int32)
    last = torch.randint(S // 2, S, (T,), generator=g, device=DEV, dtype=torch.int32)
    last[0] = -1                                         # a token that sees nothing
    out, lse = C.sparse_prefill_fp4_fwd(q, cache, idx, ks, vs, n_valid=nv, block_size=bs, last_slot=last)
    torch.cuda.synchronize()
    ref = reference(q, cache, ks, vs, idx, nv, block_size=bs, last_slot=last)
    assert compare(out, lse, ref, f"blocks {bs}") >= 24


def test_large_tiny_and_hot_queries(C):
    """Magnitudes far outside FP16's range, an all-zero head, and scores of
    +-10^3 whose running maximum rises tile after tile."""
    T, S = 7, 700
    q, cache, ks, vs, g = case(C, T, S, (12, 1), seed=21, spread=1.0)
    q[1] *= 1e-30
    q[2] *= 1e-3
    q[3, 5, 7] = 3000.0
    q[4, 2] = 0.0
    q[5] *= 300.0
    idx = W.random_lists(T, 1, 600, S, g, DEV)
    k = torch.from_numpy(R.fp4_rows(cache.buffer)[0][:, 0]).to(DEV)
    score = k[idx[5, 0].long()] @ q[5, 0].double()
    idx[5, 0] = idx[5, 0, score.argsort()]               # ascending scores for head 0
    out, lse = C.sparse_prefill_fp4_fwd(q, cache, idx, ks, vs)
    torch.cuda.synchronize()
    compare(out, lse, reference(q, cache, ks, vs, idx), "range")


def test_nan_reaches_only_what_it_must(C):
    T, S = 4, 300
    q, cache, ks, vs, g = case(C, T, S, (6, 1), seed=33)
    idx = W.random_lists(T, 1, 200, S - 2, g, DEV)
    want, wl = C.sparse_prefill_fp4_fwd(q, cache, idx, ks, vs)
    bad = cache.buffer.clone()
    bad[S - 2:, 0, 256:] = 0x7f                          # NaN scales in rows no live entry names
    nv = torch.full((T, 1), 200, dtype=torch.int32, device=DEV)
    lists = torch.cat((idx, torch.full((T, 1, 9), S - 1, dtype=torch.int32, device=DEV)), 2)
    out, lse = C.sparse_prefill_fp4_fwd(q, C.Fp4Cache(bad), lists, ks, vs, n_valid=nv)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)
    # one V block scale: NaN in its 16 dims of the tokens that name the row
    bad = cache.buffer.clone()
    slot = int(idx[1, 0, 150])
    bad[slot, 0, 272 + 3] = 0x7f
    out, lse = C.sparse_prefill_fp4_fwd(q, C.Fp4Cache(bad), idx, ks, vs)
    torch.cuda.synchronize()
    hit = (idx[:, 0] == slot).any(1).cpu().numpy()
    assert hit[1]
    o = R.f64(out)
    assert np.all(np.isnan(o[hit][..., 48:64]))
    assert np.isfinite(np.delete(o[hit], np.s_[48:64], -1)).all() and np.isfinite(o[~hit]).all()
    assert torch.equal(lse, wl)
    # a NaN query element: that head alone
    q2 = q.clone()
    q2[2, 3, 9] = float("nan")
    out, lse = C.sparse_prefill_fp4_fwd(q2, cache, idx, ks, vs)
    torch.cuda.synchronize()
    o, l = R.f64(out), R.f64(lse)
    assert np.isnan(o[2, 3]).all() and np.isnan(l[2, 3])
    keep = np.ones(o.shape[:2], dtype=bool)
    keep[2, 3] = False
    assert np.array_equal(o[keep], R.f64(want)[keep])


def test_strides(C):
    """Q, out and lists as strided views, head-major cache rows, one list shared by the heads."""
    T, S, heads = 6, 500, (24, 2)
    q, cache, ks, vs, g = case(C, T, S, heads, seed=41)
    wide = torch.zeros((T, 40, 256), dtype=torch.bfloat16, device=DEV)
    wide[:, 8:32] = q
    hm = cache.buffer.transpose(0, 1).contiguous().transpose(0, 1)
    idx = W.random_lists(T, 1, 300, S, g, DEV).expand(T, 2, 300)
    o = torch.full((T, 30, 256), 9.0, dtype=torch.bfloat16, device=DEV)
    l = torch.full((T, 50), 9.0, device=DEV)
    C.sparse_prefill_fp4_fwd(wide[:, 8:32], C.Fp4Cache(hm), idx, ks, vs, out=o[:, 3:27], lse=l[:, :24])
    torch.cuda.synchronize()
    compare(o[:, 3:27].contiguous(), l[:, :24].contiguous(), reference(q, cache, ks, vs, idx), "strides")
    assert bool((o[:, :3] == 9).all()) and bool((o[:, 27:] == 9).all()) and bool((l[:, 24:] == 9).all())
    # every head of the query the same row
    same = q[:, :1].expand(T, 24, 256)
    out, lse = C.sparse_prefill_fp4_fwd(same, cache, idx, ks, vs)
    torch.cuda.synchronize()
    compare(out, lse, reference(same.contiguous(), cache, ks, vs, idx), "broadcast query")


def test_far_slots(C):
    """Row offsets past 2^31 bytes."""
    S = 7_600_000
    q, near, ks, vs, g = case(C, 2, 64, (6, 1), seed=51)
    cache = C.fp4_cache(S, 1, DEV)
    cache.buffer[-64:] = near.buffer
    idx = torch.arange(64, dtype=torch.int32, device=DEV).repeat(2, 1, 1)
    want, wl = C.sparse_prefill_fp4_fwd(q, near, idx, ks, vs)
    out, lse = C.sparse_prefill_fp4_fwd(q, cache, idx + (S - 64), ks, vs)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("heads", [(24, 2), (16, 2)])
@pytest.mark.parametrize("T,splits", [(6, 0), (6, 1), (6, 3), (6, 16), (7, 6), (40, 3)])
def test_split_k_decode(C, heads, T, splits):
    """One chunk, chunks merged in a cluster (where they fit) and through the workspace."""
    ctx, K = 700, 650
    q, cache, ks, vs, g = case(C, T, T * ctx, heads, seed=61)
    idx = W.random_lists(T, 2, K, ctx, g, DEV) + (torch.arange(T, dtype=torch.int32, device=DEV) * ctx).view(T, 1, 1)
    nv = torch.full((T, 2), K, dtype=torch.int32, device=DEV)
    nv[1], nv[2], nv[3, 0] = 0, 300, 1
    need = C.decode_fp4_workspace_bytes(q, cache, idx, splits)
    ws = torch.full((need + 256,), 0xff, dtype=torch.uint8, device=DEV)
    out, lse = C.sparse_decode_fp4_fwd(q, cache, idx, ks, vs, n_valid=nv, num_splits=splits, workspace=ws)
    torch.cuda.synchronize()
    assert compare(out, lse, reference(q, cache, ks, vs, idx, nv), f"decode splits={splits}") == heads[0]
    again, _ = C.sparse_decode_fp4_fwd(q, cache, idx, ks, vs, n_valid=nv, num_splits=splits)
    torch.cuda.synchronize()
    assert torch.equal(again, out)


@pytest.mark.parametrize("heads", [(24, 2), (16, 2)])
@pytest.mark.parametrize("T,K", [(1, 256), (3, 257), (16, 384), (24, 384), (24, 512), (40, 500), (8, 2048), (24, 1024)])
def test_automatic_chunks(C, heads, T, K):
    """The chunks that are picked for short and long lists, with and without room for clusters."""
    ctx = K + 52
    q, cache, ks, vs, g = case(C, T, T * ctx, heads, seed=T + K)
    idx = W.random_lists(T, 2, K, ctx, g, DEV) + (torch.arange(T, dtype=torch.int32, device=DEV) * ctx).view(T, 1, 1)
    nv = torch.full((T, 2), K, dtype=torch.int32, device=DEV)
    nv[T // 2, 0], nv[T - 1, 1] = 130, 0
    need = C.decode_fp4_workspace_bytes(q, cache, idx)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
    out, lse = C.sparse_decode_fp4_fwd(q, cache, idx, ks, vs, n_valid=nv, workspace=ws)
    torch.cuda.synchronize()
    t = sorted({0, T // 2, T - 1})
    ti = torch.tensor(t)
    assert compare(out[ti], lse[ti], reference(q, cache, ks, vs, idx, nv, tokens=t), f"T={T} K={K}") == heads[0] // 2


def test_workspace_belongs_to_the_launching_stream(C):
    """An allocated workspace is let go on return, with its kernels still to run:
    only work of the same stream may be given its memory."""
    heads, T, ctx, K = (24, 2), 40, 700, 650           # 240 chunks: more than run at once
    q, cache, ks, vs, g = case(C, T, T * ctx, heads, seed=62)
    idx = W.random_lists(T, 2, K, ctx, g, DEV) + (torch.arange(T, dtype=torch.int32, device=DEV) * ctx).view(T, 1, 1)
    assert C.decode_fp4_workspace_bytes(q, cache, idx, 3) > 0
    want, wl = C.sparse_decode_fp4_fwd(q, cache, idx, ks, vs, num_splits=3)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    held = lambda: sum(x["total_size"] for x in torch.cuda.memory_snapshot() if x["stream"] == side.cuda_stream)
    before = held()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = C.sparse_decode_fp4_fwd(q, cache, idx, ks, vs, num_splits=3, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert held() > before
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_allocated_workspace_in_a_graph(C):
    """A captured call that allocates its workspace and outputs: replays give what an eager call gives."""
    heads, T, ctx, K = (24, 2), 40, 400, 380
    q, cache, ks, vs, g = case(C, T, T * ctx, heads, seed=64)
    base = (torch.arange(T, dtype=torch.int32, device=DEV) * ctx).view(T, 1, 1)
    lists = [W.random_lists(T, 2, K, ctx, g, DEV) + base for _ in "ab"]
    assert C.decode_fp4_workspace_bytes(q, cache, lists[0], 3) > 0
    call = lambda idx: C.sparse_decode_fp4_fwd(q, cache, idx, ks, vs, num_splits=3)
    want = [call(idx) for idx in lists]
    idx = lists[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = call(idx)
    for i in (1, 0):
        idx.copy_(lists[i])
        junk = torch.full((1 << 22,), float("nan"), device=DEV)  # eager memory between the replays
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1]) and bool(junk.isnan().all())


def test_signs_repeats_and_ranges(C):
    """Negative tensor scales, a row named more than once, and integers past 32 bits."""
    T, S, heads = 5, 400, (24, 2)
    q, cache, ks, vs, g = case(C, T, S, heads, seed=63)
    idx = W.random_lists(T, 2, 300, S, g, DEV)
    idx[:, :, 200:] = idx[:, :, :100]
    idx[1] = 17
    for a, b in ((ks, vs), (-ks, vs), (ks, -vs)):
        for f in (C.sparse_prefill_fp4_fwd, C.sparse_decode_fp4_fwd):
            out, lse = f(q, cache, idx, a, b)
            torch.cuda.synchronize()
            compare(out, lse, reference(q, cache, a, b, idx), f"{f.__name__} {a} {b}")
    with pytest.raises(ValueError):
        C.sparse_prefill_fp4_fwd(q, cache, idx, ks, vs, block_size=(1 << 32) + 1)
    with pytest.raises(ValueError):
        C.sparse_decode_fp4_fwd(q, cache, idx, ks, vs, num_splits=1 << 32)


def test_append_then_decode(C):
    """The run of a serving step: rows appended, then attention whose lists name
    them, captured once and replayed with other contents."""
    B, ctx, heads, K, S = 5, 300, (16, 2), 200, 1500
    table = C.rope_table(ctx, 64, base=1e6, device=DEV)

    def inputs(seed):
        q, cache, ks, vs, g = case(C, B, S, heads, seed)
        k, v = (torch.randn((B, 2, 256), generator=g, device=DEV).to(torch.bfloat16) for _ in "kv")
        pos = torch.randint(K, ctx, (B,), generator=g, device=DEV, dtype=torch.int32)
        base = torch.arange(B, device=DEV, dtype=torch.int32) * ctx
        idx = W.random_lists(B, 2, K, K, g, DEV) + base.view(B, 1, 1)
        idx[:, :, 7] = (base + pos).view(B, 1)           # the token itself
        return q, k, v, pos, base + pos, cache.buffer, idx, ks, vs

    a, b = inputs(71), inputs(72)
    buf = [x.clone() if isinstance(x, torch.Tensor) else x for x in a]
    q, k, v, pos, slots, rows, idx, ks, vs = buf
    cache = C.Fp4Cache(rows)
    qr, out = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty(q.shape[:2], device=DEV)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)

    def step():
        C.kv_append_fp4(k, v, pos, slots, table, cache, ks, vs, q=q, q_out=qr)
        C.sparse_decode_fp4_fwd(qr, cache, idx, ks, vs, workspace=ws, out=out, lse=lse)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x in (b, a):
        for d, src in zip(buf[:7], x[:7]):
            d.copy_(src)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        p = x[3].cpu().numpy()
        tab = R.f64(table)
        # the query as the definition rotates it, rounded once to BF16
        qd = R.rotate(R.f64(x[0]), tab, p, 64)
        assert np.all(np.abs(R.f64(qr) - qd) <= 2.0 ** -8 * np.abs(qd) + 2.0 ** -20)
        kd, vd = R.fp4_rows(x[5])
        for part, y, ts in ((kd, R.rotate(R.f64(x[1]), tab, p, 64), ks), (vd, R.f64(x[2]), vs)):
            _, _, val = R.fp4_encode(y, ts)
            part[x[4].cpu().numpy()] = val / np.float64(np.float32(ts))
        kd, vd = kd * np.float64(np.float32(ks)), vd * np.float64(np.float32(vs))
        compare(out, lse, reference_rows(qr, kd, vd, x[6]), "step")
