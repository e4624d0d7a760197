"""Plain definitions, in numpy, of the operators next to the expert products:
balanced routing, the int8 row quantiser and product, and the block norms.
Sums and choices in 64 bits; where the definition fixes a chain of fp32
operations, that chain."""
import numpy as np

SOFTMAX, SIGMOID = 0, 1
PLAIN, SILU, GELU = -1, 0, 1


def route(z, k, bias=None, scale=None, scoring=SOFTMAX, n_group=1, topk_group=1, group_top=1,
          renorm=True, factor=1.0):
    """(ids [T,k] int64, w [T,k] float64, load [E] int64)."""
    z = np.minimum(np.asarray(z, np.float32), np.finfo(np.float32).max).astype(np.float64)
    T, E = z.shape
    avail = z > -np.inf  # False for NaN
    zz = np.where(avail, z, 0.0)
    if scoring == SIGMOID:
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-zz))
    else:
        top = np.max(np.where(avail, zz, -np.inf), axis=1, keepdims=True, initial=-np.inf)
        e = np.exp(zz - np.where(np.isfinite(top), top, 0.0)) * avail
        den = e.sum(axis=1, keepdims=True)
        s = e / np.where(den > 0, den, 1.0)
    s = np.where(avail, s, 0.0)
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    with np.errstate(invalid="ignore"):
        c = np.where(avail, s + b, -np.inf)
    c = np.where(np.isnan(c), -np.inf, np.minimum(c, np.finfo(np.float64).max))
    ranked = c.copy()
    inside = np.ones((T, E), bool)
    if n_group > 1:
        gs = E // n_group
        best = -np.sort(-c.reshape(T, n_group, gs), axis=2)[:, :, :group_top]
        with np.errstate(over="ignore"):
            score = best.sum(axis=2)
        order = np.argsort(-score, axis=1, kind="stable")[:, :topk_group]
        kept = np.zeros((T, n_group), bool)
        np.put_along_axis(kept, order, True, axis=1)
        inside = np.repeat(kept, gs, axis=1)
    # outside the kept groups after everything, unavailable ones included
    order = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -ranked, ~inside), axis=1)
    ids = order[:, :k]
    chosen = np.take_along_axis(s, ids, 1)
    chosen = np.where(np.take_along_axis(c, ids, 1) > -np.inf, chosen, 0.0)
    w = chosen
    if renorm:
        den = chosen.sum(axis=1, keepdims=True)
        w = np.where(den > 0, chosen / np.where(den > 0, den, 1.0), 0.0)
    w = w * float(np.float32(factor))
    if scale is not None:
        w = w * np.asarray(scale, np.float64)[ids]
    return ids, w, np.bincount(ids.reshape(-1), minlength=E)


def quantize_i8(v):
    """fp32 values of bf16 rows -> (codes int8, scales fp32), IEEE fp32 steps."""
    v = np.asarray(v, np.float32)
    amax = np.abs(v).max(axis=1)  # NaN propagates
    s = np.where(amax == 0, np.float32(1), amax / np.float32(127)).astype(np.float32)
    with np.errstate(invalid="ignore"):
        q = np.rint(v / s[:, None])
    q = np.clip(np.where(np.isnan(q), 0, q), -127, 127)
    return q.astype(np.int8), s


def act64(act, g):
    if act == SILU:
        with np.errstate(over="ignore"):
            return g / (1.0 + np.exp(-g))
    # 0.5 (1 + tanh v) = 1 / (1 + e^-2v), which does not cancel at large negative v
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-2.0 * np.sqrt(2.0 / np.pi) * (g + 0.044715 * g ** 3)))


def linear_i8(x, xs, w, ws, act=PLAIN):
    """Plain: the fp32 result of the definition's steps (exact to the bit).
    Gated: in float64 from those fp32 gate and up values."""
    acc = x.astype(np.float64) @ w.astype(np.float64).T  # exact: below 2^53
    m = np.asarray(xs, np.float32)[:, None] * np.asarray(ws, np.float32)[None, :]
    v = acc.astype(np.float32) * m
    if act == PLAIN:
        return v
    I = w.shape[0] // 2
    return act64(act, v[:, :I].astype(np.float64)) * v[:, I:].astype(np.float64)


def to_bf16(v):
    """fp32 array rounded to bf16 (nearest, ties to even), as fp32 values."""
    u = np.ascontiguousarray(v, np.float32).view(np.uint32)
    r = ((u.astype(np.uint64) + 0x7fff + ((u >> 16) & 1)) & 0xffff0000).astype(np.uint32)
    return np.where(np.isnan(v), np.float32(np.nan), r.view(np.float32))


def _inv_rms(v, eps):
    mean = (v.astype(np.float64) ** 2).mean(axis=1).astype(np.float32)
    return (np.float32(1) / np.sqrt(mean + np.float32(eps)))[:, None]


def block_norm(r, y=None, post_w=None, gate=None, token_gate=None, alpha=1.0, beta=1.0,
               post_eps=1e-6, pre_w=None, pre_eps=1e-6):
    """The fp32 steps of the definition on fp32 arrays of bf16 values:
    (r_out or None, a or None), fp32 arrays of bf16 values."""
    r = np.asarray(r, np.float32)
    r_out = a = None
    if y is not None:
        t = np.asarray(y, np.float32)
        if post_w is not None:
            t = (t * _inv_rms(t, post_eps)) * post_w
        if gate is not None:
            t = t * gate
        m = np.float32(beta)
        if token_gate is not None:
            m = m * np.asarray(token_gate, np.float32)[:, None]
        r_out = r = to_bf16(np.float32(alpha) * r + m * t)
    if pre_w is not None:
        a = to_bf16((r * _inv_rms(r, pre_eps)) * pre_w)
    return r_out, a


def block_norm64(r, y=None, post_w=None, gate=None, token_gate=None, alpha=1.0, beta=1.0,
                 post_eps=1e-6):
    """The new residual's formula in float64, unrounded."""
    d = np.float64
    t = np.asarray(y, d)
    if post_w is not None:
        t = t / np.sqrt((t * t).mean(axis=1, keepdims=True) + post_eps) * np.asarray(post_w, d)
    if gate is not None:
        t = t * np.asarray(gate, d)
    m = beta if token_gate is None else beta * np.asarray(token_gate, d)[:, None]
    return alpha * np.asarray(r, d), m * t
