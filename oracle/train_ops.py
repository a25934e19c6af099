"""fp64 restatement of the training-step operators: 8-bit activation checkpoints and the weight gradient
taken from them, the norms around a block with its gate and residual scales, token log probabilities.
Test infrastructure only; written from the formulas, shares no code with the library."""

from __future__ import annotations

import numpy as np

BLOCK = 32


# ---------------------------------------------------------------- checkpoints
def ckpt_layout(rows: int, cols: int):
    """(bytes of a row of q, bytes of a row of scales, offset of the scales, bytes in all)."""
    ld_q = (cols + 31) // 32 * 32
    ld_e = (ld_q // 32 + 15) // 16 * 16
    at = (rows * ld_q + 127) // 128 * 128
    return ld_q, ld_e, at, at + rows * ld_e


def ckpt_encode(x: np.ndarray):
    """q (rows x ld_q int8, zeros past cols) and scale bytes (rows x ld_q/32), x as float64 of float32 values."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    ld_q = ckpt_layout(rows, cols)[0]
    w = np.zeros((rows, ld_q))
    w[:, :cols] = x
    w = w.reshape(rows, -1, BLOCK)
    q = np.zeros(w.shape, np.int8)
    b = np.zeros(w.shape[:2], np.uint8)
    for r in range(rows):
        for k in range(w.shape[1]):
            v = w[r, k]
            if not np.all(np.isfinite(v)):
                b[r, k] = 255
                continue
            a, e = np.abs(v).max(), -126
            while a > 127.0 * 2.0 ** e:
                e += 1
            most = 63 if e >= 122 else 127
            q[r, k] = np.clip(np.rint(v * 2.0 ** -e), -most, most)
            b[r, k] = e + 127
    return q.reshape(rows, ld_q), b


def ckpt_decode(q: np.ndarray, b: np.ndarray, cols: int) -> np.ndarray:
    s = np.where(b == 255, np.nan, 2.0 ** (b.astype(np.float64) - 127))
    return (q.astype(np.float64) * np.repeat(s, BLOCK, axis=1))[:, :cols]


def ckpt_split(buf: np.ndarray, rows: int, cols: int):
    """q and scale bytes of a checkpoint buffer (uint8)."""
    ld_q, ld_e, at, n = ckpt_layout(rows, cols)
    q = buf[:rows * ld_q].view(np.int8).reshape(rows, ld_q)
    return q, buf[at:n].reshape(rows, ld_e)[:, :ld_q // BLOCK]


def wgrad(dy: np.ndarray, xhat: np.ndarray, add=None) -> np.ndarray:
    dw = np.asarray(dy, np.float64).T @ np.asarray(xhat, np.float64)
    return dw if add is None else dw + add


# ---------------------------------------------------------------- norms around a block
def gate_act(g, act: str):
    """act(g) and its slope."""
    g = np.asarray(g, np.float64)
    s = 1 / (1 + np.exp(-g))
    if act == "identity":
        return g, np.ones_like(g)
    if act == "sigmoid":
        return s, s * (1 - s)
    return g * s, s + g * s * (1 - s)


def norm_fwd(h, y, w_post=None, w_pre=None, gate=None, act="identity", h_scale=1.0, y_scale=1.0, eps=1e-6, post=True,
             pre=True) -> dict:
    h, y = np.asarray(h, np.float64), np.asarray(y, np.float64)
    cols = h.shape[1]
    r_post = 1 / np.sqrt((y * y).sum(1) / cols + eps)
    n = y * r_post[:, None] * (1.0 if w_post is None else w_post) if post else y
    h2 = h_scale * h + y_scale * (1.0 if gate is None else gate_act(gate, act)[0]) * n
    r_pre = 1 / np.sqrt((h2 * h2).sum(1) / cols + eps)
    return dict(h=h2, x=h2 * r_pre[:, None] * (1.0 if w_pre is None else w_pre) if pre else None, r_post=r_post,
                r_pre=r_pre, n=n)


def norm_bwd(h2, y, dx, dh_in, r_post, r_pre, w_post=None, w_pre=None, gate=None, act="identity", h_scale=1.0,
             y_scale=1.0, post=True, pre=True) -> dict:
    """Gradients of norm_fwd; h2 is its h.  dgate is per element (sum it over rows for a channel gate)."""
    h2, y = np.asarray(h2, np.float64), np.asarray(y, np.float64)
    d = np.zeros_like(h2) if dh_in is None else np.array(dh_in, np.float64)
    out = {}
    if pre:
        hh = h2 * np.asarray(r_pre, np.float64)[:, None]
        out["dw_pre"] = (dx * hh).sum(0)
        g = dx * (1.0 if w_pre is None else w_pre)
        d = d + np.asarray(r_pre, np.float64)[:, None] * (g - hh * (g * hh).mean(1, keepdims=True))
    out["dh"] = h_scale * d
    value, slope = (1.0, 0.0) if gate is None else gate_act(gate, act)
    yh = y * np.asarray(r_post, np.float64)[:, None] if post else y
    n = yh * (1.0 if w_post is None or not post else w_post)
    out["dgate"] = y_scale * slope * n * d
    dn = y_scale * value * d
    if post:
        out["dw_post"] = (dn * yh).sum(0)
        g = dn * (1.0 if w_post is None else w_post)
        out["dy"] = np.asarray(r_post, np.float64)[:, None] * (g - yh * (g * yh).mean(1, keepdims=True))
    else:
        out["dy"] = dn
    return out


# ---------------------------------------------------------------- token log probabilities
def _z(x, inv_temp):
    """logits * inv_temp; past the range of fp32 it counts as infinite."""
    z = x * inv_temp
    most = float(np.finfo(np.float32).max)
    return np.where(z < -most, -np.inf, np.where(z > most, np.inf, z))


def _log_p(z):
    """Log probabilities from the distance to the maximum (z - lse would lose the sum beside a large maximum)."""
    d = z - z.max()
    return d - np.log(np.exp(d).sum())


def logp_fwd(logits, targets, inv_temp=1.0, top_k=0) -> dict:
    """Rows of nothing but masked entries (-inf or a type's lowest value): lse -inf, logp -inf (0 without a target), entropy 0, top log probabilities -inf."""
    x = np.asarray(logits, np.float64)
    rows, vocab = x.shape
    out = dict(logp=np.zeros(rows), entropy=np.zeros(rows), lse=np.zeros(rows),
               ids=np.zeros((rows, top_k), np.int64), top=np.zeros((rows, top_k)))
    for r in range(rows):
        z = _z(x[r], inv_temp)
        t = int(targets[r])
        if np.isnan(z).any() or (z == np.inf).any():
            lse = entropy = np.nan
            lp = np.full(vocab, np.nan)
        elif x[r].max() <= -1e37 or (z == -np.inf).all():
            lse, entropy, lp = -np.inf, 0.0, np.full(vocab, -np.inf)
        else:
            lp = _log_p(z)
            lse = z.max() + np.log(np.exp(z - z.max()).sum())
            p = np.exp(lp)
            entropy = -(p[p > 0] * lp[p > 0]).sum()
        out["lse"][r], out["entropy"][r] = lse, entropy
        out["logp"][r] = 0.0 if t < 0 else np.nan if t >= vocab else lp[t]
        order = sorted(range(vocab), key=lambda j: (np.isnan(x[r, j]), -x[r, j] if not np.isnan(x[r, j]) else 0.0, j))
        out["ids"][r] = order[:top_k]
        out["top"][r] = lp[order[:top_k]]
    return out


def logp_bwd(logits, targets, g_logp=None, g_entropy=None, inv_temp=1.0) -> np.ndarray:
    x = np.asarray(logits, np.float64)
    f = logp_fwd(x, targets, inv_temp)
    d = np.zeros_like(x)
    for r in range(x.shape[0]):
        if f["lse"][r] == -np.inf:
            continue
        t = int(targets[r])
        lp = _log_p(_z(x[r], inv_temp))
        p = np.exp(lp)
        if g_logp is not None and t >= 0:
            if t >= x.shape[1]:
                d[r] = np.nan
                continue
            d[r] -= g_logp[r] * p
            d[r, t] += g_logp[r]
        if g_entropy is not None:
            d[r] -= g_entropy[r] * np.where(p > 0, p * (np.where(p > 0, lp, 0.0) + f["entropy"][r]), 0.0)
    return d * inv_temp
