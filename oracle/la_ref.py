"""Linear attention with a decay for each head in float64 (numpy), by its definition: one token
after the other, the gradients as the adjoint of that recurrence.  Test infrastructure only; the
HIP library shares no code with it.

    S_t = e^{g_t} S_{t-1} + k_t v_tᵀ        o_t = scale · S_tᵀ q_t

q, k [B, T, Hk, dk]; v, o [B, T, H, dv]; g None, [H] or [B, T, H]; s0 [B, H, dk, dv] or None;
lengths None or [B]: tokens at and behind a row's length change nothing, and their outputs and
gradients are 0.
"""
import numpy as np


def _operands(q, k, v, g, s0, lengths):
    v = np.asarray(v, np.float64)
    B, T, H, dv = v.shape
    rep = H // q.shape[2]
    q = np.repeat(np.asarray(q, np.float64), rep, axis=2)
    k = np.repeat(np.asarray(k, np.float64), rep, axis=2)
    a = np.ones((B, T, H))
    if g is not None:
        with np.errstate(under="ignore"):
            a = a * np.exp(np.asarray(g, np.float64))
    n = np.full(B, T) if lengths is None else np.clip(np.asarray(lengths, np.int64), 0, T)
    live = np.arange(T)[None] < n[:, None]
    # behind the end: whatever stands there (NaN too) is replaced, not multiplied
    q, k, v = (np.where(live[..., None, None], x, 0.0) for x in (q, k, v))
    a = np.where(live[..., None], a, 1.0)
    s = np.zeros((B, H, q.shape[3], dv)) if s0 is None else np.array(s0, np.float64)
    return q, k, v, a, live, s


def fwd(q, k, v, g=None, s0=None, scale=1.0, lengths=None):
    """o [B, T, H, dv], s_final [B, H, dk, dv]."""
    q, k, v, a, live, s = _operands(q, k, v, g, s0, lengths)
    o = np.zeros(v.shape)
    for t in range(v.shape[1]):
        s = a[:, t, :, None, None] * s + k[:, t, :, :, None] * v[:, t, :, None, :]
        o[:, t] = scale * np.einsum("bhi,bhij->bhj", q[:, t], s)
    return np.where(live[..., None, None], o, 0.0), s


def bwd(q, k, v, do, g=None, s0=None, ds_final=None, scale=1.0, lengths=None):
    """Gradients of sum(do·o) + sum(ds_final·s_final): dict dq, dk, dv, dg, ds0."""
    Hk = q.shape[2]
    q, k, v, a, live, s = _operands(q, k, v, g, s0, lengths)
    do = np.where(live[..., None, None], np.asarray(do, np.float64), 0.0)
    B, T, H, _ = v.shape
    states = [s]
    for t in range(T):
        states.append(a[:, t, :, None, None] * states[-1] + k[:, t, :, :, None] * v[:, t, :, None, :])
    r = np.zeros_like(s) if ds_final is None else np.array(ds_final, np.float64)
    dq, dk, dv, dg = (np.zeros_like(x) for x in (q, k, v, a))
    for t in reversed(range(T)):
        r = r + scale * q[:, t, :, :, None] * do[:, t, :, None, :]
        dq[:, t] = scale * np.einsum("bhij,bhj->bhi", states[t + 1], do[:, t])
        dk[:, t] = np.einsum("bhij,bhj->bhi", r, v[:, t])
        dv[:, t] = np.einsum("bhij,bhi->bhj", r, k[:, t])
        da = np.einsum("bhij,bhij->bh", r, states[t])
        dg[:, t] = a[:, t] * da
        r = a[:, t, :, None, None] * r
    m = live[..., None, None]
    dq, dk, dv = np.where(m, dq, 0.0), np.where(m, dk, 0.0), np.where(m, dv, 0.0)
    dg = np.where(live[..., None], dg, 0.0)
    fold = lambda x: x.reshape(B, T, Hk, H // Hk, -1).sum(3)  # noqa: E731
    if g is None:
        dg = None
    elif np.ndim(g) == 1:
        dg = dg.sum((0, 1))
    return dict(dq=fold(dq), dk=fold(dk), dv=dv, dg=dg, ds0=None if s0 is None else r)
