"""RMS norm with the residual's addition, and products with 4-bit weights, in float64 (numpy), by
their definitions.  Test infrastructure only; the HIP library shares no code with it."""
import numpy as np


def rms_fwd(x, w, res=None, eps=1e-5):
    """y, r (both float64, unrounded)."""
    r = np.asarray(x, np.float64)
    if res is not None:
        r = r + np.asarray(res, np.float64)
    return r / np.sqrt((r * r).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64), r


def rms_bwd(dy, r, w, dr=None, eps=1e-5):
    """dx, dw: y_i = w_i r_i m^-1/2 with m = mean(r²) + eps, so
    dL/dr_j = w_j dy_j m^-1/2 - r_j m^-3/2 / D · Σ_i w_i dy_i r_i."""
    dy, r, w = (np.asarray(a, np.float64) for a in (dy, r, w))
    m = (r * r).mean(-1, keepdims=True) + eps
    dx = w * dy * m ** -0.5 - r * m ** -1.5 / r.shape[-1] * (w * dy * r).sum(-1, keepdims=True)
    if dr is not None:
        dx = dx + np.asarray(dr, np.float64)
    return dx, (dy * r * m ** -0.5).reshape(-1, r.shape[-1]).sum(0)


def q4_weights(wq, scales, zeros, group):
    """W [N, K] from codes [N, K / 2] (low half first), scales and zeros [N, ceil(K / group)]."""
    wq = np.asarray(wq)
    u = np.empty((wq.shape[0], 2 * wq.shape[1]))
    u[:, 0::2] = wq % 16
    u[:, 1::2] = wq // 16
    at = np.arange(u.shape[1]) // group
    z = 8.0 if zeros is None else np.asarray(zeros, np.float64)[:, at]
    return (u - z) * np.asarray(scales, np.float64)[:, at]


def q4_mv(x, wq, scales, zeros=None, group=128, x_scale=None):
    y = np.asarray(x, np.float64) @ q4_weights(wq, scales, zeros, group).T
    return y if x_scale is None else y * np.asarray(x_scale, np.float64)[..., None]
