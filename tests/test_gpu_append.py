"""Cache appends with position rotation against plain FP64 definitions.

Tolerances, derived: a BF16 result is one rounding (half a step: 2^-8
relative) of a rotation whose FP32 arithmetic rounds twice (2^-23 of the two
products' magnitudes).  An E4M3 byte is within half a step (2^-4 relative, or
half of the subnormal step 2^-9) of y / ts, which FP32 arithmetic moves by
less than 2^-21 of the two products' magnitudes.  4-bit rows are decided
exactly and compared byte for byte.
"""
import numpy as np
import pytest
import torch

import cache_ref as R
from parity import host

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = "cuda"
FORMATS = ("bf16", "fp8", "fp4")
KS, VS = 4.7 / 2688, 5.1 / 2688


@pytest.fixture(scope="module")
def C():
    from top_sparse_attention_qsa_b200 import _capi
    return _capi


def case(C, T, heads, rot, S, seed, P=None, packed=True):
    """q, k, v as views of one packed projection [T, Hq + 2 Hkv, 256], a table, positions, distinct slots."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    Hq, Hkv = heads
    x = torch.randn((T, Hq + 2 * Hkv, 256), generator=g, device=DEV).to(torch.bfloat16)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    P = P or 5000
    table = C.rope_table(P, rot, base=1e6, device=DEV)
    pos = torch.randint(0, P, (T,), generator=g, device=DEV, dtype=torch.int32)
    slots = torch.randperm(S, generator=g, device=DEV)[:T].to(torch.int32)
    return q, k, v, table, pos, slots


def new_cache(C, fmt, S, Hkv):
    """Caches filled with a pattern, so that a row nobody named shows a stray write."""
    if fmt == "fp4":
        return (C.Fp4Cache(torch.full((S, Hkv, 288), 0x5a, dtype=torch.uint8, device=DEV)),)
    kc = torch.full((S, Hkv, 256 * (2 if fmt == "bf16" else 1)), 0x5a, dtype=torch.uint8, device=DEV)
    dt = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
    return kc.view(dt), kc.clone().view(dt)


def call(C, fmt, cache, k, v, pos, slots, table, **kw):
    if fmt == "bf16":
        return C.kv_append(k, v, pos, slots, table, *cache, **kw), None, None
    if fmt == "fp8":
        return C.kv_append_fp8(k, v, pos, slots, table, *cache, KS, VS, want_seen=True, **kw)
    return C.kv_append_fp4(k, v, pos, slots, table, cache[0], KS, VS, want_seen=True, **kw)


def check_rotated(got, want, mag, label):
    d = np.abs(R.f64(got) - want)
    tol = 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -15) + 2.0 ** -23 * mag * 1.01 + 2.0 ** -134
    assert np.all(d <= tol), f"{label}: {d.max()}"


def magnitude(x, table, pos, rot, inter):
    """|x_a c| + |x_b s| of every element, the scale of the rotation's roundings."""
    y = np.abs(x)
    t = np.abs(table)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        c, s = t[pos, i][:, None], t[pos, rot // 2 + i][:, None]
        xa, xb = np.abs(x[..., a]), np.abs(x[..., b])
        y[..., a], y[..., b] = xa * c + xb * s, xb * c + xa * s
    return y


def check(fmt, cache, before, q_out, seen, q, k, v, table, pos, slots, rot, inter, S, valid=None):
    """Every output against the definitions; `valid` [T]: the position is inside the table."""
    T = k.shape[0]
    tab, p = R.f64(table) if rot else np.zeros((1, 0)), pos.cpu().numpy() if rot else np.zeros(T, dtype=int)
    valid = np.ones(T, dtype=bool) if valid is None else valid
    p = np.where(valid, p, 0)
    kx, vx = R.f64(k), R.f64(v)
    ky = R.rotate(kx, tab, p, rot, inter)
    km = magnitude(kx, tab, p, rot, inter)
    if q is not None:
        qx = R.f64(q)
        qy = R.rotate(qx, tab, p, rot, inter)
        qm = magnitude(qx, tab, p, rot, inter)
        check_rotated(q_out[torch.from_numpy(valid)], qy[valid], qm[valid], "q")
    sl = slots.cpu().numpy()
    put = (sl >= 0) & (sl < S) & valid
    rows = sl[put]
    other = np.ones(S, dtype=bool)
    other[rows] = False
    if fmt == "fp4":
        now, was = host(cache[0].buffer).numpy(), host(before[0].buffer).numpy()
        assert np.array_equal(now[other], was[other])
        for part, y, ts in ((0, ky, KS), (1, vx, VS)):
            code, e, val = R.fp4_encode(y, ts)
            want = code[..., 0::2] + 16 * code[..., 1::2]
            assert np.array_equal(now[rows][..., 128 * part:128 * part + 128], want[put]), "codes"
            wb = torch.from_numpy(e).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            assert np.array_equal(now[rows][..., 256 + 16 * part:272 + 16 * part], wb[put]), "block scales"
            got = R.f64(seen[part])[valid]
            # the value in FP32 (one rounding), then BF16
            assert np.all(np.abs(got - val[valid]) <= 2.0 ** -8 * (1 + 2.0 ** -14) * np.abs(val[valid]))
        return
    for part, y, m, ts in ((0, ky, km, KS), (1, vx, np.abs(vx) * 0, VS)):
        now, was = host(cache[part]), host(before[part])
        u8 = lambda x: x.view(torch.uint8).numpy()  # noqa: E731
        assert np.array_equal(u8(now)[other], u8(was)[other])
        got = R.f64(now[torch.from_numpy(rows.astype(np.int64))])
        if fmt == "bf16":
            check_rotated(torch.from_numpy(got), y[put], m[put], "cache")
            continue
        want = np.clip(y / np.float64(np.float32(ts)), -448, 448)
        tol = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + 2.0 ** -21 * (np.abs(want) + m / ts)
        assert np.all(np.abs(got - want[put]) <= tol[put])
        sv = R.f64(seen[part])[valid]
        full = np.zeros_like(y)
        full[put] = got
        d = np.abs(sv - full[valid] * np.float64(np.float32(ts)))[put[valid]]
        assert np.all(d <= 2.0 ** -8 * (1 + 2.0 ** -14) * np.abs(full[valid] * ts)[put[valid]])


def clone(cache):
    return tuple(type(c)(c.buffer.clone()) if hasattr(c, "buffer") else c.clone() for c in cache)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heads,rot,inter", [((3, 1), 64, False), ((24, 2), 64, True), ((16, 2), 256, False),
                                             ((12, 1), 16, True), ((6, 1), 0, False), ((5, 3), 144, False)])
@pytest.mark.parametrize("T", [1, 37])
def test_formats(C, fmt, heads, rot, inter, T):
    S = 101
    q, k, v, table, pos, slots = case(C, T, heads, max(rot, 2), S, seed=T + rot)
    if rot == 0:
        table, pos = None, None
    cache = new_cache(C, fmt, S, heads[1])
    before = clone(cache)
    q_out, ks, vs = call(C, fmt, cache, k, v, pos, slots, table, q=q, interleaved=inter)
    torch.cuda.synchronize()
    check(fmt, cache, before, q_out, (ks, vs), q, k, v, table, pos, slots, rot, inter, S)


@pytest.mark.parametrize("heads,rot,inter", [((9, 2), 80, False), ((17, 1), 256, False), ((41, 7), 112, True),
                                             ((8, 4), 0, False), ((25, 5), 256, True)])
def test_shares_of_the_warps(C, heads, rot, inter):
    """Head counts that do not divide into a warp's rows, rotary widths that are not powers of two."""
    S, T = 64, 11
    q, k, v, table, pos, slots = case(C, T, heads, max(rot, 2), S, seed=rot + heads[0])
    if rot == 0:
        table, pos = None, None
    cache = new_cache(C, "bf16", S, heads[1])
    before = clone(cache)
    q_out, _, _ = call(C, "bf16", cache, k, v, pos, slots, table, q=q, interleaved=inter)
    torch.cuda.synchronize()
    check("bf16", cache, before, q_out, (None, None), q, k, v, table, pos, slots, rot, inter, S)
    got = C.kv_append(k, v, pos, slots, table, *cache, q=q, q_out=q, interleaved=inter)
    torch.cuda.synchronize()
    assert torch.equal(got, q_out)


@pytest.mark.parametrize("fmt", FORMATS)
def test_padding_bad_slots_and_positions(C, fmt):
    T, S = 40, 77
    q, k, v, table, pos, slots = case(C, T, (6, 1), 64, S, seed=3)
    slots[5] = -1
    slots[9] = S
    slots[10] = 2 ** 31 - 1
    slots[30:] = -7
    pos[2], pos[3] = -1, 5000
    valid = np.ones(T, dtype=bool)
    valid[[2, 3]] = False
    cache = new_cache(C, fmt, S, 1)
    before = clone(cache)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out = torch.full_like(q, 7.0)
    _, ks, vs = call(C, fmt, cache, k, v, pos, slots, table, q=q, q_out=q_out, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == C.STATUS_OOB_SLOT | C.STATUS_BAD_POSITION
    assert bool((q_out[2:4] == 7.0).all())
    check(fmt, cache, before, q_out, (ks, vs), q, k, v, table, pos, slots, 64, False, S, valid)
    status.zero_()
    slots[9] = slots[10] = -1
    pos[2:4] = 0
    call(C, fmt, cache, k, v, pos, slots, table, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_no_query_no_tokens_no_slots(C, fmt):
    S = 19
    q, k, v, table, pos, slots = case(C, 7, (3, 1), 64, S, seed=5)
    cache = new_cache(C, fmt, S, 1)
    before = clone(cache)
    none, ks, vs = call(C, fmt, cache, k, v, pos, slots, table)
    assert none is None
    torch.cuda.synchronize()
    check(fmt, cache, before, None, (ks, vs), None, k, v, table, pos, slots, 64, False, S)
    before = clone(cache)
    call(C, fmt, cache, k[:0], v[:0], pos[:0], slots[:0], table, q=q[:0])
    torch.cuda.synchronize()
    for a, b in zip(cache, before):
        a, b = getattr(a, "buffer", a), getattr(b, "buffer", b)
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("rot,inter", [(64, False), (256, True)])
def test_query_in_place(C, rot, inter):
    q, k, v, table, pos, slots = case(C, 33, (24, 2), rot, 50, seed=9)
    cache = new_cache(C, "bf16", 50, 2)
    want = C.kv_append(k, v, pos, slots, table, *cache, q=q, interleaved=inter)
    got = C.kv_append(k, v, pos, slots, table, *cache, q=q, q_out=q, interleaved=inter)
    torch.cuda.synchronize()
    assert got.data_ptr() == q.data_ptr() and torch.equal(want, q)


def test_fp4_borders(C):
    """Values exactly on the E2M1 midpoints, one BF16 step beside them, blocks
    whose scale underflows or saturates, signed zeros."""
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]
    rows = []
    for s in (1.0, 2.0 ** -3, 1.125, 3.5, 2.0 ** 6):
        for eps in (-2.0 ** -7, 0.0, 2.0 ** -7):
            blk = np.zeros(16)
            blk[:8] = np.array(mids) * s * (1 + np.array([eps] * 7 + [0]))
            blk[8:15] = -blk[:7]
            blk[15] = 6 * s
            rows.append(blk)
    rows.append(np.zeros(16))
    rows.append(-np.zeros(16))
    rows.append(np.full(16, 2.0 ** -20))                 # scale rounds to zero
    rows.append(np.full(16, 3e4))                        # scale saturates at 448
    rows.append(np.linspace(-448 * 6, 448 * 6, 16))
    while len(rows) % 16:
        rows.append(np.linspace(-1, 1, 16) * len(rows))
    y = np.stack(rows).reshape(-1, 1, 256)
    x = torch.from_numpy(y).to(torch.bfloat16).to(DEV)
    T = x.shape[0]
    for ts in (1.0, 0.7, 2.0 ** -9):
        cache = C.fp4_cache(T, 1, DEV)
        C.kv_append_fp4(x, x, None, torch.arange(T, dtype=torch.int32, device=DEV), None, cache, ts, ts)
        torch.cuda.synchronize()
        code, e, _ = R.fp4_encode(R.f64(x), ts)
        b = host(cache.buffer).numpy()
        for part in range(2):
            assert np.array_equal(b[..., 128 * part:128 * part + 128], code[..., 0::2] + 16 * code[..., 1::2])
            assert np.array_equal(R.f64((cache.k_bscale, cache.v_bscale)[part]), e)


def test_non_finite_values(C):
    """NaN stays NaN in the cache, infinities saturate; other blocks and rows are as without them."""
    q, k, v, table, pos, slots = case(C, 6, (3, 1), 64, 8, seed=13, packed=False)
    v[1, 0, 40] = float("nan")
    v[2, 0, 200] = float("inf")
    v[3, 0, 100] = float("-inf")
    cache = new_cache(C, "fp4", 8, 1)
    _, _, seen = call(C, "fp4", cache, k, v, pos, slots, table)
    torch.cuda.synchronize()
    s = R.f64(seen)
    e = R.f64(cache[0].v_bscale)[slots.cpu().numpy(), 0]
    assert np.all(np.isnan(s[1, 0, 32:48])) and np.isfinite(np.delete(s[1, 0], np.s_[32:48])).all()
    assert np.isnan(e[1, 2]) and e[2, 12] == 448 and e[3, 6] == 448
    assert s[2, 0, 200] > 0 and s[3, 0, 100] < 0 and np.isfinite(s[2:4]).all()
    assert abs(s[2, 0, 200] / (6 * 448 * VS) - 1) < 2.0 ** -8
    c8 = new_cache(C, "fp8", 8, 1)
    _, _, seen = call(C, "fp8", c8, k, v, pos, slots, table)
    torch.cuda.synchronize()
    s = R.f64(seen)
    assert np.isnan(s[1, 0, 40]) and np.isnan(s).sum() == 1
    assert abs(s[2, 0, 200] / (448 * VS) - 1) < 2.0 ** -8 and s[3, 0, 100] < 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_far_slots(C, fmt):
    """Row offsets past 2^31 bytes."""
    S = {"bf16": 4300000, "fp8": 8500000, "fp4": 7600000}[fmt]
    q, k, v, table, pos, _ = case(C, 3, (3, 1), 64, 16, seed=21)
    slots = torch.tensor([S - 1, 0, S - 2], dtype=torch.int32, device=DEV)
    if fmt == "fp4":
        cache = (C.fp4_cache(S, 1, DEV),)
        tail = (C.Fp4Cache(cache[0].buffer[-2:]),)
    else:
        dt = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
        cache = tuple(torch.zeros((S, 1, 256), dtype=torch.uint8 if fmt == "fp8" else dt, device=DEV).view(dt) for _ in "kv")
        tail = tuple(c[-2:] for c in cache)
    _, ks, vs = call(C, fmt, cache, k, v, pos, slots, table)
    torch.cuda.synchronize()
    small = new_cache(C, fmt, 2, 1)
    sl = torch.tensor([1, -1, 0], dtype=torch.int32, device=DEV)
    call(C, fmt, small, k, v, pos, sl, table)
    torch.cuda.synchronize()
    for a, b in zip(tail, small):
        a, b = getattr(a, "buffer", a), getattr(b, "buffer", b)
        assert torch.equal(a.contiguous().view(torch.uint8), b.view(torch.uint8))


def test_graph_and_side_stream(C):
    """Captured once, replayed on new contents; the same on another stream."""
    T, S = 21, 64
    a = case(C, T, (6, 1), 64, S, seed=31, packed=False)
    b = case(C, T, (6, 1), 64, S, seed=32, packed=False)
    cache = C.fp4_cache(S, 1, DEV)
    qo = torch.empty_like(a[0])
    buf = [x.clone() for x in a]
    fn = lambda: C.kv_append_fp4(buf[1], buf[2], buf[4], buf[5], buf[3], cache, KS, VS, q=buf[0], q_out=qo)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    for x in (b, a):
        for d, src in zip(buf, x):
            d.copy_(src)
        cache.buffer.zero_()
        g.replay()
        want = C.fp4_cache(S, 1, DEV)
        wq, _, _ = C.kv_append_fp4(x[1], x[2], x[4], x[5], x[3], want, KS, VS, q=x[0])
        torch.cuda.synchronize()
        assert torch.equal(cache.buffer, want.buffer) and torch.equal(qo, wq)
