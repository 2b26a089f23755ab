"""Plain definitions of the cache formats, in FP64 with numpy: the rotation,
the E4M3 and E2M1 roundings, the 4-bit rows and attention over them.  Shares
no code with the library."""
import numpy as np
import torch

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
F = np.float32


def f64(x):
    return x.detach().cpu().to(torch.float64).numpy()


def rotate(x, table, positions, R, interleaved=False):
    """x [T, H, 256] float64 rotated by table[positions] [T, >= R] (cosines, then sines)."""
    y = np.array(x)
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        c = table[positions, i][:, None]
        s = table[positions, R // 2 + i][:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def e4m3(x):
    """Nearest E4M3 value (ties to even, saturating at 448)."""
    a = np.abs(x)
    e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    step = np.exp2(np.maximum(e, -6) - 3)
    return np.sign(x) * np.minimum(np.round(a / step) * step, 448.0)


def block_scales(y, ts):
    """E4M3 block scales of y [..., 256]: [..., 16] float64."""
    amax = np.abs(y).reshape(*y.shape[:-1], 16, 16).max(-1).astype(F)
    return e4m3((amax * (F(1) / (F(6) * F(ts)))).astype(np.float64))


def fp4_encode(y, ts):
    """codes [..., 256] (0..15), block scales [..., 16], values [..., 256]."""
    e = block_scales(y, ts)
    step = np.repeat(e, 16, -1) * float(F(ts))
    a = np.abs(y)
    dist = np.abs(a[..., None] - MAGNITUDES * step[..., None])
    dist = dist[..., [0, 2, 4, 6, 1, 3, 5, 7]]           # even codes first: a tie goes to them
    code = np.array([0, 2, 4, 6, 1, 3, 5, 7])[dist.argmin(-1)]
    code = np.where(step > 0, code, 0)
    neg = np.signbit(y)
    return code + 8 * neg, e, np.where(neg, -1.0, 1.0) * MAGNITUDES[code] * step


def fp4_rows(buffer):
    """(k values / k_scale, v values / v_scale) [S, Hkv, 256] float64 of a cache buffer [S, Hkv, 288] uint8."""
    b = buffer.detach().cpu()
    out = []
    for part in range(2):
        by = b[..., 128 * part:128 * part + 128].numpy().astype(np.int64)
        code = np.stack((by & 15, by >> 4), -1).reshape(*by.shape[:-1], 256)
        e = f64(b[..., 256 + 16 * part:272 + 16 * part].contiguous().view(torch.float8_e4m3fn))
        val = np.where(code & 8, -1.0, 1.0) * MAGNITUDES[code & 7]
        out.append(val * np.repeat(e, 16, -1))
    return out


def fp4_buffer(S, Hkv, seed, device, spread=1.0):
    """A cache buffer of standard normal keys and values (K times `spread`), with the tensor scales."""
    g = np.random.default_rng(seed)
    ts = 4.6 / 2688
    buf = np.zeros((S, Hkv, 288), dtype=np.uint8)
    for part, std in ((0, spread), (1, 1.0)):
        code, e, _ = fp4_encode(g.standard_normal((S, Hkv, 256)) * std, ts * std)
        buf[..., 128 * part:128 * part + 128] = code[..., 0::2] + 16 * code[..., 1::2]
        buf[..., 256 + 16 * part:272 + 16 * part] = torch.from_numpy(e).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return torch.from_numpy(buf).to(device), ts * spread, ts


def attention(q, k, v, idx, n_valid=None, scale=1 / 16, block_size=1, last_slot=None, tokens=None):
    """FP64 attention over lists: q [T, Hq, 256], k and v [S, Hkv, 256] float64 arrays, idx [T, Hkv, K] int tensor.
    Returns (out [n, Hq, 256], lse [n, Hq])."""
    qn, ix = f64(q), idx.cpu().numpy().astype(np.int64)
    T, Hq, _ = qn.shape
    S, Hkv, _ = k.shape
    G = Hq // Hkv
    nv = None if n_valid is None else n_valid.cpu().numpy()
    last = None if last_slot is None else last_slot.cpu().numpy()
    tokens = range(T) if tokens is None else tokens
    out = np.zeros((len(tokens), Hq, 256))
    lse = np.full((len(tokens), Hq), -np.inf)
    for r, t in enumerate(tokens):
        for g in range(Hkv):
            e = ix[t, g]
            if nv is not None:
                e = e[:max(0, int(nv[t, g]))]
            e = e[(e >= 0) & (e * block_size < S)]
            rows = (e[:, None] * block_size + np.arange(block_size)).reshape(-1)
            rows = rows[rows < S]
            if last is not None:
                rows = rows[rows <= last[t]]
            if rows.size == 0:
                continue
            z = scale * (qn[t, g * G:(g + 1) * G] @ k[rows, g].T)
            m = z.max(-1, keepdims=True)
            p = np.exp(z - m)
            l = p.sum(-1, keepdims=True)
            out[r, g * G:(g + 1) * G] = (p / l) @ v[rows, g]
            lse[r, g * G:(g + 1) * G] = (m + np.log(l))[:, 0]
    return out, lse
