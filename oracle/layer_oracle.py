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
