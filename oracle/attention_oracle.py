"""Plain float64 reference of the attention-side operators (numpy, CPU): head
norms with rotary positions and their gradient, the 8-bit paged cache, and
attention over it. Written from the definitions, one row, page or sequence at a
time; shares no code with the GPU path. Test infrastructure only."""
import numpy as np


# ---- head norms and rotary positions ------------------------------------------

def _pairs(rot, layout):
    i = np.arange(rot // 2)
    return (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)


def rotate(n, positions, table, layout, back=False):
    """n [T, H, D] with the pairs of its first table.shape[1] elements turned."""
    rot = table.shape[1]
    a, b = _pairs(rot, layout)
    row = table.astype(np.float64)[positions]
    c, s = row[:, None, :rot // 2], row[:, None, rot // 2:]
    if back:
        s = -s
    y = n.astype(np.float64).copy()
    y[..., a] = n[..., a] * c - n[..., b] * s
    y[..., b] = n[..., b] * c + n[..., a] * s
    return y


def norm_rope(x, positions, table, weight=None, norm=True, eps=1e-6, layout="half"):
    n = x.astype(np.float64)
    if norm:
        n = n / np.sqrt((n * n).mean(-1, keepdims=True) + eps)
        if weight is not None:
            n = n * weight
    return n if table is None else rotate(n, positions, table, layout)


def norm_rope_backward(x, g, positions, table, weight=None, norm=True, eps=1e-6, layout="half"):
    """(g_x, g_weight) for g the gradient of norm_rope's output."""
    gn = g.astype(np.float64)
    if table is not None:
        gn = rotate(gn, positions, table, layout, back=True)
    if not norm:
        return gn, None
    x = x.astype(np.float64)
    D = x.shape[-1]
    root = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    w = np.ones(D) if weight is None else weight.astype(np.float64)
    # y_i = w_i x_i / root, droot/dx_j = x_j / (D root)
    u = gn * w
    gx = u / root - x * (u * x).sum(-1, keepdims=True) / (D * root ** 3)
    return gx, (gn * x / root).sum((0, 1))


# ---- the 8-bit cache -------------------------------------------------------------

class Cache:
    """Keys and values [pages, heads, page, dim] int8 (values token-major here)
    and their scales, in the fp32 arithmetic the format is defined by."""

    def __init__(self, n_pages, heads, page, dim):
        self.page = page
        self.keys = np.zeros((n_pages, heads, page, dim), np.int8)
        self.values = np.zeros((n_pages, heads, page, dim), np.int8)
        self.k_scale = np.zeros((n_pages, heads), np.float32)
        self.v_scale = np.zeros((n_pages, heads), np.float32)

    def append(self, block_table, start, k, v):
        """k, v [n, heads, dim] float32 after the first `start` tokens of the
        sequence whose pages block_table (a row) names."""
        n, at = k.shape[0], 0
        while at < n:
            pos = start + at
            page, held = block_table[pos // self.page], pos % self.page
            m = min(self.page - held, n - at)
            for pool, scale, x in ((self.keys, self.k_scale, k), (self.values, self.v_scale, v)):
                for h in range(x.shape[1]):
                    self._store(pool[page, h], scale, (page, h), held, x[at:at + m, h].astype(np.float32))
            at += m

    @staticmethod
    def _store(entries, scale, key, held, x):
        with np.errstate(all="ignore"):
            s = np.abs(x).max() / np.float32(127) if np.isfinite(x).all() else np.float32(np.nan)
            if held:
                old = scale[key]
                new = old if np.isnan(old) or s <= old else s
                if not np.isnan(new) and new > old:
                    ratio = np.float32(old / new)
                    entries[:held] = np.rint(entries[:held].astype(np.float32) * ratio).astype(np.int8)
                s = new
            q = np.rint(x / s) if s > 0 else np.zeros_like(x)
            entries[held:held + len(x)] = np.clip(np.nan_to_num(q), -127, 127).astype(np.int8)
            scale[key] = s

    def read(self, block_table, start, end):
        """Tokens start .. end - 1 as float32: (k, v) [n, heads, dim]."""
        pos = np.arange(start, end)
        pages, slots = np.asarray(block_table)[pos // self.page], pos % self.page
        k = self.keys[pages, :, slots].astype(np.float32) * self.k_scale[pages][..., None]
        v = self.values[pages, :, slots].astype(np.float32) * self.v_scale[pages][..., None]
        return k, v


# ---- attention ---------------------------------------------------------------------

def attend(q, k, v, p0, scale, window=0):
    """q [n, H, D] at positions p0 .. p0 + n - 1 over k, v [L, K, D]. Returns
    out, lse, and for error bounds sum_j p_j |v_j| and the largest
    scale sum_d |q_d k_jd| of each row's keys."""
    n, H, D = q.shape
    L, K, _ = k.shape
    q, k, v = (t.astype(np.float64) for t in (q, k, v))
    out, weight = np.zeros((n, H, D)), np.zeros((n, H, D))
    lse, size = np.full((n, H), -np.inf), np.zeros((n, H))
    for i in range(n):
        p = p0 + i
        lo = max(0, p - window + 1) if window else 0
        if p < lo:
            continue
        for h in range(H):
            kh, vh = k[lo:p + 1, h // (H // K)], v[lo:p + 1, h // (H // K)]
            s = scale * (kh @ q[i, h])
            m = s.max()
            e = np.exp(s - m)
            w = e / e.sum()
            out[i, h], weight[i, h] = w @ vh, w @ np.abs(vh)
            lse[i, h] = m + np.log(e.sum())
            size[i, h] = abs(scale) * (np.abs(kh) @ np.abs(q[i, h])).max()
    return out, lse, weight, size
