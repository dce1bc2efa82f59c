"""fp64 numpy oracle of the dense gated FFN and what stands around an FFN: the norms before and after a
block with its gate and residual sum, and AdamW with fp32 or 8-bit
moments.  Test infrastructure only; written from the formulas."""
import numpy as np

ADAMW_BLOCK = 256


def _per_block(scale, n):
    return np.repeat(np.asarray(scale, dtype=np.float64), ADAMW_BLOCK)[:n]


def adamw_m_value(code, scale):
    """m held in int8 codes: scale * c * |c|, one scale per block of 256."""
    c = np.asarray(code, dtype=np.float64)
    return c * np.abs(c) * _per_block(scale, c.size)


def adamw_v_value(code, scale):
    """v held in uint8 codes: (scale * c^2)^2."""
    c = np.asarray(code, dtype=np.float64)
    return (c * c * _per_block(scale, c.size)) ** 2


def adamw_positions(value, most):
    """Where non-negative magnitudes lie between the codes 0..most (before
    rounding), and the scale of each block."""
    n = value.size
    nb = -(-n // ADAMW_BLOCK)
    full = np.zeros(nb * ADAMW_BLOCK)
    full[:n] = value
    top = full.reshape(nb, ADAMW_BLOCK).max(1)
    each = _per_block(top, n)
    pos = np.where(each > 0, most * np.sqrt(value / np.where(each > 0, each, 1.0)), 0.0)
    return pos, top / most ** 2


def adamw(p, g, m, v, *, lr, beta1, beta2, eps, step, weight_decay=0.0, grad_scale=1.0):
    """New p, m, v and the size of the update's terms (for error bounds)."""
    g = grad_scale * g
    m_new = beta1 * m + (1 - beta1) * g
    v_new = beta2 * v + (1 - beta2) * g * g
    den = np.sqrt(v_new / (1 - beta2 ** step)) + eps
    size = lr / (1 - beta1 ** step)
    terms = size * (np.abs(beta1 * m) + np.abs((1 - beta1) * g)) / den
    return p * (1 - lr * weight_decay) - size * m_new / den, m_new, v_new, terms


def norm_forward(y, r, w_post, gate, w_pre, *, gate_group=0, a=1.0, s=1.0, eps=1e-6):
    """r', n and the rows' inverse norms; None where an argument is None."""
    T = r.shape[0]
    p = q = n = None
    if y is None:
        out = r
    else:
        o = y
        if w_post is not None:
            p = 1 / np.sqrt(np.mean(y * y, axis=1) + eps)
            o = y * p[:, None] * w_post
        if gate is not None:
            o = gate[np.arange(T) // gate_group] * o
        out = a * r + s * o
    if w_pre is not None:
        q = 1 / np.sqrt(np.mean(out * out, axis=1) + eps)
        n = out * q[:, None] * w_pre
    return out, n, p, q


def norm_backward(dn, dr_out, y, r_out, w_post, gate, w_pre, p, q, *, gate_group=0, a=1.0, s=1.0):
    """Gradients (dict) from the kept inverse norms p (post) and q (pre)."""
    T, d = (r_out if r_out is not None else dr_out).shape
    out = {}
    G = np.zeros((T, d)) if dr_out is None else dr_out.copy()
    if dn is not None:
        rh = r_out * q[:, None]
        e = dn * w_pre
        G = G + q[:, None] * (e - rh * np.mean(e * rh, axis=1, keepdims=True))
        out["dw_pre"] = np.sum(dn * rh, axis=0)
    out["G"] = G
    if y is None:
        out["dr"] = G
        return out
    out["dr"] = a * G
    row = np.arange(T) // gate_group if gate is not None else None
    k = s * G if gate is None else s * gate[row] * G
    yh = y if w_post is None else y * p[:, None]
    o = yh if w_post is None else yh * w_post
    if w_post is None:
        out["dy"] = k
    else:
        f = k * w_post
        out["dy"] = p[:, None] * (f - yh * np.mean(f * yh, axis=1, keepdims=True))
        out["dw_post"] = np.sum(k * yh, axis=0)
    if gate is not None:
        out["dgate"] = np.zeros_like(gate)
        np.add.at(out["dgate"], row, s * G * o)
    return out


def activation(name, z):
    """act(z) and act'(z)."""
    from scipy.special import expit, ndtr
    if name == "relu":
        return np.maximum(z, 0.0), (z > 0).astype(np.float64)
    if name == "silu":
        p = expit(z)
        return z * p, p * (1 + z * (1 - p))
    if name == "gelu":
        return z * ndtr(z), ndtr(z) + z * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
    c = np.sqrt(2 / np.pi)
    t = np.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def gated_ffn(x, Wg, Wu, Wd, act):
    """z, u, h, y of the dense gated FFN; weights [F, d]."""
    z, u = x @ Wg.T, x @ Wu.T
    h = activation(act, z)[0] * u
    return z, u, h, h @ Wd


def gated_ffn_backward(x, dy, Wg, Wu, Wd, act, z, u):
    """Gradients from z and u: dict of h, dh, du, dz, dx, dWg, dWu, dWd."""
    a, da = activation(act, z)
    h, dh = a * u, dy @ Wd.T
    du, dz = dh * a, dh * u * da
    return dict(h=h, dh=dh, du=du, dz=dz, dx=du @ Wu + dz @ Wg, dWg=dz.T @ x, dWu=du.T @ x,
                dWd=h.T @ dy)
