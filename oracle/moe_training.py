"""Float64 oracle of the rest of a training step: the balance loss with its gradient, the linear
router's backward pass for a dense gradient, the gradient norm, and the AdamW step with its
8-bit moments. Written from the definitions in include/moe.h, with plain numpy.
"""
from __future__ import annotations

import numpy as np

M32 = np.uint64(0xFFFFFFFF)
ADAMW_BLOCK = 128


def balance_loss(logits, topk_idx, token_mask=None, alpha=1e-2, z_coef=0.0, d_loss=1.0) -> dict:
    """counts, n_tokens, prob_mean, loss (balance + z, balance, z) and d_logits."""
    T, N = logits.shape
    keep = np.ones(T, bool) if token_mask is None else np.asarray(token_mask) != 0
    n = int(keep.sum())
    counts = np.zeros(N, np.int64)
    prob_mean, d_logits = np.zeros(N), np.zeros((T, N))
    if n == 0:
        return dict(counts=counts, n_tokens=0, prob_mean=prob_mean, loss=np.zeros(3), d_logits=d_logits)
    chosen = topk_idx[keep].reshape(-1)
    counts = np.bincount(chosen[(chosen >= 0) & (chosen < N)], minlength=N)
    L = np.asarray(logits, np.float64)[keep]
    some = np.isfinite(L).any(1)  # a row of -inf only adds nothing
    p, lse = np.zeros_like(L), np.zeros(n)
    m = L[some].max(1, keepdims=True)
    e = np.exp(L[some] - m)
    p[some] = e / e.sum(1, keepdims=True)
    lse[some] = (m + np.log(e.sum(1, keepdims=True)))[:, 0]
    f = counts / n
    prob_mean = p.sum(0) / n
    balance, z = alpha * N * float(f @ prob_mean), z_coef * float((lse ** 2).sum()) / n
    d_logits[keep] = d_loss * p * (alpha * N / n * (f - (p @ f)[:, None]) + (2 * z_coef / n * lse)[:, None])
    return dict(counts=counts, n_tokens=n, prob_mean=prob_mean, loss=np.array([balance + z, balance, z]),
                d_logits=d_logits)


def router_backward(x, w_router, d_logits) -> dict:
    """Gradients of L = x W_r^T + b."""
    return dict(d_x=d_logits @ w_router, d_w_router=d_logits.T @ x, d_logit_bias=d_logits.sum(0))


def grad_norm(grads, max_norm):
    norm = float(np.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads)))
    return norm, (min(1.0, max_norm / (norm + 1e-6)) if np.isfinite(norm) else float("nan"))


# ---------------------------------------------------------------- AdamW
def _mix(x):
    x = x & M32
    x ^= x >> np.uint64(16)
    x = (x * np.uint64(0x2F5A6B1D)) & M32
    x ^= x >> np.uint64(15)
    x = (x * np.uint64(0xB4C3D7A9)) & M32
    return x ^ (x >> np.uint64(16))


def random_bits(n, seed, step, index, first=0):
    """Three 16-bit words for elements first .. first + n of the tensor at `index` of the list:
    those that round m, sqrt(v) and the parameter."""
    u = lambda v: np.uint64(v & 0xFFFFFFFF)
    i = np.arange(first, first + n, dtype=np.uint64)
    with np.errstate(over="ignore"):
        key = _mix(_mix(np.array([u(index * 0x632BE5AB + seed)])) + u(step * 0x9E3779B1))[0]
        h = _mix((i & M32) * u(0x9E3779B1) + key + (i >> np.uint64(32)) * u(0x85EBCA6B))
        h2 = (h * u(0xD1B54A35) + key) & M32
    return (h & np.uint64(0xFFFF)).astype(np.int64), (h >> np.uint64(16)).astype(np.int64), \
        (h2 >> np.uint64(16)).astype(np.int64)


def round_up_by_chance(x, digits, lowest, u):
    """x on the grid of `digits` binary digits after the first (spacing at least 2**lowest), its
    magnitude rounded up where the part cut off plus u (in [0, 1)) reaches one spacing."""
    a = np.abs(x)
    e = np.frexp(a)[1] - 1.0
    grid = np.exp2(np.maximum(e - digits, float(lowest)))
    return np.sign(x) * np.floor(a / grid + u) * grid


def quantise_moment(x, bits, keep_nonzero):
    """(values of the codes, scales): E4M3 codes in float64, one scale per ADAMW_BLOCK elements."""
    n = x.size
    blocks = -(-n // ADAMW_BLOCK)
    pad = np.zeros(blocks * ADAMW_BLOCK)
    pad[:n] = x
    amax = np.abs(pad.reshape(blocks, ADAMW_BLOCK)).max(1)
    amax[amax < 2.0 ** -96] = 0.0
    per = np.repeat(amax, ADAMW_BLOCK)[:n]
    rel = np.divide(x * 448.0, per, out=np.zeros(n), where=per > 0)
    code = round_up_by_chance(rel, 3, -9, (bits * 16 + 8) / 2.0 ** 20)
    code = np.clip(code, -448.0, 448.0)
    if keep_nonzero:
        code = np.where((rel > 0) & (code == 0), 2.0 ** -9, code)
    return code, amax / 448.0


def adamw(param, grad, m, v, *, step, index=0, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0,
          grad_scale=1.0, seed=0, bits=32, m_scale=None, v_scale=None, bf16_alone=False) -> dict:
    """One tensor's step. param: the fp32 values (the master copy where there is one). With
    bits = 8, m and v hold the codes' values. Returns the new param, m and v before rounding
    (m_exact, v_exact) and as they are stored."""
    if bits == 8:
        m = m * np.repeat(m_scale, ADAMW_BLOCK)[:m.size]
        v = (v * np.repeat(v_scale, ADAMW_BLOCK)[:v.size]) ** 2
    g = grad * grad_scale
    b1, b2 = betas
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    update = lr / (1 - b1 ** step) * m / (np.sqrt(v) / np.sqrt(1 - b2 ** step) + eps)
    p = param * (1 - lr * weight_decay) - update
    out = dict(param_exact=p, update=update, m_exact=m, v_exact=v, param=p, m=m, v=v)
    um, uv, up = random_bits(m.size, seed, step, index)
    if bits == 8:
        out["m"], out["m_scale"] = quantise_moment(m, um, False)
        out["v"], out["v_scale"] = quantise_moment(np.sqrt(v), uv, True)
    if bf16_alone:
        out["param"] = round_up_by_chance(p, 7, -133, up / 65536.0)
    return out
