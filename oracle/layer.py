"""fp64 numpy oracle of the operators around the FFN: AdamW with fp32 or 8-bit
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
