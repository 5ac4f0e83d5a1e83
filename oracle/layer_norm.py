"""Layer norm over rows with its gradients, float64 -- TEST INFRASTRUCTURE
ONLY.

y = (x - mean) rstd w + b, rstd = 1 / sqrt(mean((x - mean)^2) + eps);
grad_x = rstd (gw - mean(gw) - xhat mean(gw xhat)), gw = g w; grad_w = sum over
rows of g xhat, grad_b = sum over rows of g.
"""

import numpy as np


def layer_norm(x, w, b, eps):
    """(y, mean, rstd) of float64 rows."""
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    rstd = 1 / np.sqrt(np.square(x - mean[:, None]).mean(1) + eps)
    return (x - mean[:, None]) * rstd[:, None] * w + b, mean, rstd


def layer_norm_grad(g, x, mean, rstd, w):
    """(grad_x, grad_w, grad_b) with the statistics as given."""
    xhat = (np.asarray(x, np.float64) - mean[:, None]) * rstd[:, None]
    gw = g * w
    grad_x = rstd[:, None] * (gw - gw.mean(1, keepdims=True) - xhat * (gw * xhat).mean(1, keepdims=True))
    return grad_x, (g * xhat).sum(0), g.sum(0)
