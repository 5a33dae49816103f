"""Plain float64 reference of the paged 4-bit cache and of attention over it (numpy, CPU),
written from the definitions; shares no code with the GPU path. Test infrastructure only."""
import numpy as np

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def decode(codes):
    """Codes 0 .. 15 as the numbers they stand for."""
    return np.where(codes & 8, -1.0, 1.0) * LEVELS[codes & 7]


def encode(q):
    """The nearest code of every quotient q, of two as near the even one; -0 keeps its sign."""
    d = np.abs(np.abs(q)[..., None] - LEVELS)
    # an even code is taken a hair nearer than it is, far less than any two quotients differ
    code = np.argmin(d * (1 + 1e-13 * (np.arange(8) % 2)), -1)
    return (code | np.where(np.signbit(q), 8, 0)).astype(np.uint8)


def unpack(b):
    return np.stack([b & 15, b >> 4], -1).reshape(b.shape[:-1] + (2 * b.shape[-1],))


def pack(codes):
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def quantise_keys(k):
    """(codes, exponents + 127) of k [..., D] fp32."""
    x = k.reshape(k.shape[:-1] + (-1, 32)).astype(np.float64)
    top = np.abs(x).max(-1)
    fine = np.isfinite(top)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.ceil(np.log2(np.where(fine & (top > 0), top, 1) / 6))
    for step in (-1, 1):            # a logarithm beside a whole number
        e = np.where((6 * 2.0 ** (e + step) >= top) & (step < 0), e + step, e)
        e = np.where((6 * 2.0 ** e < top) & (step > 0), e + step, e)
    e = np.where(top > 0, np.maximum(e, -127), -127)
    codes = encode(np.where(fine[..., None], x, 0) / 2.0 ** np.where(fine, e, 0)[..., None])
    return codes.reshape(k.shape), np.where(fine, e + 127, 255).astype(np.uint8)


def quantise_values(v):
    """(codes, scales) of v [..., D] fp32: scale and quotients are fp32."""
    v = v.astype(np.float32)
    top = np.abs(v).max(-1)
    s = np.where(np.isfinite(top), top / np.float32(6), np.float32(np.nan)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s[..., None] > 0, v / s[..., None], np.float32(0))
    return encode(np.where(np.isfinite(q), q, 0).astype(np.float64)), s


def key_values(codes, e):
    x = decode(codes).reshape(codes.shape[:-1] + (-1, 32)) * 2.0 ** (e.astype(np.float64) - 127)[..., None]
    return np.where(e == 255, np.nan, 1.0)[..., None].repeat(32, -1).reshape(codes.shape) * x.reshape(codes.shape)


def attend(q, k, v_codes, v_scale, p0, scale, window=0):
    """Rows q [n, H, D] of tokens at p0 .. over k [S, K, D], v. Returns out, lse and, for
    bounds on errors, of every row

      w   sum_j p_j |v_j| / l                       [n, H, D]
      W   sum_j (largest p sv within 127 keys of j) |entry_j| / l    [n, H, D]
      a   largest scale sum_d |q_d k_jd| of the keys seen            [n, H]
      b   the same with every |q_d| replaced by the largest of its 32 channels"""
    n, H, D = q.shape
    S, K, _ = k.shape
    out, w, W = (np.zeros((n, H, D)) for _ in range(3))
    lse, a, b = np.full((n, H), -np.inf), np.zeros((n, H)), np.zeros((n, H))
    entries = decode(v_codes)
    for i in range(n):
        lo = max(0, p0 + i - window + 1) if window else 0
        hi = min(S, p0 + i + 1)
        if hi <= lo:
            continue
        for h in range(H):
            g = h // (H // K)
            kk, c, sv = k[lo:hi, g], entries[lo:hi, g], v_scale[lo:hi, g].astype(np.float64)
            s = scale * (kk @ q[i, h])
            m = s.max()
            p = np.exp(s - m)
            l = p.sum()
            lse[i, h] = m + np.log(l)
            ps = p * sv
            out[i, h] = ps @ c / l
            w[i, h] = ps @ np.abs(c) / l
            pad = np.pad(ps, 127)
            near = np.lib.stride_tricks.sliding_window_view(pad, 255).max(-1)
            W[i, h] = near @ np.abs(c) / l
            top = np.abs(q[i, h]).reshape(-1, 32).max(1).repeat(32)
            a[i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[i, h])).max()
            b[i, h] = abs(scale) * (np.abs(kk) @ top).max()
    return out, lse, w, W, a, b
