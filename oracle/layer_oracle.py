"""Plain float64 reference of the operators between a decoder layer's halves (numpy, CPU):
the norm with the residual's addition and its gradient. Written from the definitions;
shares no code with the GPU path. Test infrastructure only."""
import numpy as np


# ---- norm ---------------------------------------------------------------------

def norm(h, w, eps):
    """Rows of h over the root of their mean square + eps, times w (None: ones)."""
    h = h.astype(np.float64)
    y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    return y if w is None else y * w


def norm_backward(h, w, g_y, g_h, eps):
    """(g_x, g_w) of sum(y g_y) + sum(h g_h)."""
    h, g_y = h.astype(np.float64), g_y.astype(np.float64)
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    u = g_y if w is None else g_y * w
    g_x = r * u - h * r ** 3 * np.mean(u * h, axis=1, keepdims=True)
    return g_x + (0.0 if g_h is None else g_h), np.sum(g_y * h * r, axis=0)


# ---- pages of a step ------------------------------------------------------------

def plan(table, kv_lens, keep_lens, new_lens, free, n_free, page, total):
    """One page and token after another. Returns (table, free, n_free, lacking, kv_lens, cu,
    positions, slots) as lists and arrays."""
    table, stack = [list(r) for r in table], list(free)
    n = n_free
    held = [max(0, x) for x in kv_lens]
    keep = held if keep_lens is None else [min(h, max(0, k)) for h, k in zip(held, keep_lens)]
    for row, h, k in zip(table, held, keep):
        for i in range(-(-k // page), min(-(-h // page), len(row))):
            if 0 <= row[i] < len(stack) and n < len(stack):
                stack[n] = row[i]
                n += 1
    lacking, cu, lens = 0, [0], []
    positions, slots = [0] * total, [-1] * total
    for row, k, m in zip(table, keep, new_lens):
        m = max(0, m)
        for i in range(-(-k // page), min(-(-(k + m) // page), len(row))):
            if n > 0:
                n -= 1
                row[i] = stack[n]
            else:
                row[i] = -1
                lacking += 1
        for j in range(m):
            t = cu[-1] + j
            if t < total:
                positions[t] = k + j
                i = (k + j) // page
                if cu[-1] + m <= total and i < len(row) and 0 <= row[i] < len(stack):
                    slots[t] = row[i] * page + (k + j) % page
        cu.append(cu[-1] + m)
        lens.append(k + m)
    return table, stack, n, lacking, lens, cu, positions, slots
