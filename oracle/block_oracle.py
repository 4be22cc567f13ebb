"""CPU oracle of the operators around the MoE layer -- TEST INFRASTRUCTURE ONLY.

Plain float64 numpy restatements of the RMS norm with its residual and 8-bit
output, the router's losses, and the gradients of norm, routing and combine.
Independent of the CUDA library, like ``moe_oracle``.  Probabilities here are
taken as exp(log p), never as a ratio of sigmoids, so rows of very negative
logits need no rescaling.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def rmsnorm(x, residual, weight, eps):
    """(h, y, rstd)."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h, h * rstd[:, None] * np.asarray(weight, np.float64), rstd


def group_scales(y, group):
    """amax / 448 of each row's column groups (the last may be narrower)."""
    return np.stack([np.abs(y[:, c:c + group]).max(axis=1) / E4M3_MAX
                     for c in range(0, y.shape[1], group)], axis=1)


def rmsnorm_backward(dy, dh, h, weight, eps):
    """(dx, dweight) of y = rmsnorm(h) * weight, plus dh."""
    h, dy, w = (np.asarray(a, np.float64) for a in (h, dy, weight))
    r = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    g = dy * w
    # d/dh of h r with dr/dh_j = -r^3 h_j / H
    dx = g * r - h * r ** 3 * (g * h).mean(axis=1, keepdims=True)
    return dx + (0.0 if dh is None else np.asarray(dh, np.float64)), (dy * h * r).sum(axis=0)


def _log_sigmoid(l):
    return np.where(l > 0, -np.log1p(np.exp(-np.abs(l))), l - np.log1p(np.exp(-np.abs(l))))


def _normalise(logp):
    """Rows of exp(logp) / sum, and the rows' log sums; (0, 0) for a row of -inf."""
    m = logp.max(axis=1, keepdims=True)
    empty = np.isneginf(m)
    m = np.where(empty, 0.0, m)
    s = np.exp(logp - m).sum(axis=1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        lse = m + np.log(s)
        p = np.exp(logp - lse)
    return np.where(empty, 0.0, p), np.where(empty, 0.0, lse)[:, 0]


def probabilities(logits, mode):
    l = np.asarray(logits, np.float64)
    with np.errstate(invalid="ignore"):
        return _normalise(l if mode == 0 else _log_sigmoid(l))[0]


def _keep(T, mask):
    return np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool)


def balance(logits, ids, mask, E, n_seq, mode):
    """dict(counts, mean_prob, valid, losses) of the E first columns."""
    T, K = ids.shape
    L = T // n_seq
    keep = _keep(T, mask)
    counts = np.zeros((n_seq, E), np.int64)
    mean_prob = np.zeros((n_seq, E))
    n = np.zeros(n_seq, np.int64)
    z = 0.0
    bal = 0.0
    for s in range(n_seq):
        rows = s * L + np.flatnonzero(keep[s * L:(s + 1) * L])
        n[s] = len(rows)
        if not len(rows):
            continue
        sel = ids[rows].ravel()
        counts[s] = np.bincount(sel[(sel >= 0) & (sel < E)], minlength=E)
        l = np.asarray(logits[rows, :E], np.float64)
        mean_prob[s] = probabilities(l, mode).sum(axis=0) / n[s]
        z += (_normalise(l)[1] ** 2).sum()
        bal += (E * counts[s] / (K * n[s]) * mean_prob[s]).sum()
    total, full = int(n.sum()), int((n > 0).sum())
    return {"counts": counts, "mean_prob": mean_prob, "valid": np.concatenate([n, [total, full]]),
            "losses": np.array([bal / max(full, 1), z / max(total, 1)])}


def routing_weights(logits, ids, mode, scale):
    """The routing weights of fixed selections, as top-K routing defines them."""
    l = np.take_along_axis(np.asarray(logits, np.float64), ids.astype(np.int64), axis=1)
    if mode == 0:
        return _normalise(l)[0]
    return scale * _normalise(_log_sigmoid(l))[0]


def route_backward(logits, ids, weights, d_weights, d_shared_gate, mask, E, n_seq, mode, scale,
                   grad_losses):
    """dlogits of sum(d_weights * weights) + sum(d_shared_gate * sigmoid(l_E)) +
    grad_losses . losses; d_weights, d_shared_gate and grad_losses may be None."""
    T, K = ids.shape
    L = T // n_seq
    keep = _keep(T, mask)
    l = np.asarray(logits, np.float64)
    out = np.zeros((T, E + (d_shared_gate is not None)))
    stat = balance(np.where(keep[:, None], l, 0.0), ids, mask, E, n_seq, mode)
    with np.errstate(over="ignore"):
        tail = 1.0 / (1.0 + np.exp(l))  # 1 - sigmoid
    for t in np.flatnonzero(keep):
        s = t // L
        row = np.zeros(E)
        if grad_losses is not None:
            n, total, full = stat["valid"][s], stat["valid"][-2], stat["valid"][-1]
            a = grad_losses[0] * E * stat["counts"][s] / (K * n * n * full)
            p = probabilities(l[t:t + 1, :E], mode)[0]
            row += p * (a - (a * p).sum()) * (1.0 if mode == 0 else tail[t, :E])
            q, lse = _normalise(l[t:t + 1, :E])
            row += 2.0 * grad_losses[1] * lse[0] * q[0] / total
        if d_weights is not None:
            w, g = np.asarray(weights[t], np.float64), np.asarray(d_weights[t], np.float64)
            dot = (w * g).sum() / (1.0 if mode == 0 else scale)
            for k in range(K):
                e = ids[t, k]
                if 0 <= e < E:
                    row[e] += w[k] * (g[k] - dot) * (1.0 if mode == 0 else tail[t, e])
        out[t, :E] = row
        if d_shared_gate is not None:
            out[t, E] = d_shared_gate[t] * tail[t, E] * (1.0 - tail[t, E])
    return out


def unpermute_backward(dout, y, flat_to_row, weights, shared_y=None, shared_gate=None):
    """dict(dy, d_weights[, d_shared_y, d_shared_gate]); dy rows without a replica are NaN."""
    dout, y = np.asarray(dout, np.float64), np.asarray(y, np.float64)
    T, K = weights.shape
    dy = np.full(y.shape, np.nan)
    dw = np.zeros((T, K))
    for t in range(T):
        for k in range(K):
            r = flat_to_row[t * K + k]
            if 0 <= r < T * K:
                dy[r] = float(weights[t, k]) * dout[t]
                dw[t, k] = dout[t] @ y[r]
    out = {"dy": dy, "d_weights": dw}
    if shared_y is not None:
        out["d_shared_y"] = np.asarray(shared_gate, np.float64)[:, None] * dout
        out["d_shared_gate"] = (dout * np.asarray(shared_y, np.float64)).sum(axis=1)
    return out


def pack_q8(x):
    """(values / scale before their rounding to e4m3, scales) per row and 128 columns."""
    x = np.asarray(x, np.float64)
    s = group_scales(x, 128)
    wide = np.repeat(s, 128, axis=1)[:, :x.shape[1]]
    return np.divide(x, wide, out=np.zeros_like(x), where=wide > 0), s


def experts_backward(x, dout, ids, weights, w1, w3, w2, errors=None):
    """Gradients of out[t] = sum_k weights[t, k] W2[e] (silu(W1[e] x_t) * (W3[e] x_t)), e = ids[t, k]
    (below 0: dropped): dict(dx, d_weights, dw1, dw3, dw2).

    errors = (u, b): the same dict holds, under "e_" + name, how far a computation may be off
    whose matrix products sum in fp32 (half step u) and round dg, du, weights * act to bf16
    (half step b); the outputs' own rounding is not in it.
    """
    x, dout, weights = (np.asarray(a, np.float64) for a in (x, dout, weights))
    T, K = ids.shape
    E, I, H = w1.shape
    u, b = errors or (0.0, 0.0)
    out = {"dx": np.zeros((T, H)), "d_weights": np.zeros((T, K)), "dw1": np.zeros((E, I, H)),
           "dw3": np.zeros((E, I, H)), "dw2": np.zeros((E, H, I))}
    err = {k: np.zeros_like(v) for k, v in out.items()}
    # the error of a sum of n products: an addition for each 8 of them (and some for a step's
    # own alignment), each off by a step at most
    dot = lambda n: (n / 4 + 64) * u  # noqa: E731
    for e in range(E):
        t, k = np.nonzero(ids == e)
        if not len(t):
            continue
        m1, m3, m2 = (np.asarray(m[e], np.float64) for m in (w1, w3, w2))
        xe, de, w = x[t], dout[t], weights[t, k][:, None]
        g, up, a = xe @ m1.T, xe @ m3.T, de @ m2
        s = 1.0 / (1.0 + np.exp(-g))
        h, f = g * s, s * (1 + g * (1 - s))
        dg, du, act = w * a * up * f, w * a * h, w * h * up
        out["d_weights"][t, k] = (a * h * up).sum(axis=1)
        np.add.at(out["dx"], t, dg @ m1 + du @ m3)
        out["dw1"][e], out["dw3"][e], out["dw2"][e] = dg.T @ xe, du.T @ xe, de.T @ act
        if errors is None:
            continue
        A = np.abs
        # of the recomputed products; |silu'| <= 1.1, |silu''| <= 0.5; 2^-18 for exp and the few
        # products around it
        eg, eu, ea = dot(H) * (A(xe) @ A(m1).T), dot(H) * (A(xe) @ A(m3).T), dot(H) * (A(de) @ A(m2))
        near, c = 2.0 ** -18, b + 2.0 ** -18
        edg = A(w) * (A(up * f) * ea + A(a * f) * eu + 0.5 * A(a * up) * eg
                      + near * A(a * up) * (s + A(h))) + c * A(dg)
        edu = A(w) * (A(h) * ea + 1.1 * A(a) * eg) + c * A(du)
        eact = A(w) * (A(h) * eu + 1.1 * A(up) * eg) + c * A(act)
        err["d_weights"][t, k] = (A(h * up) * ea + A(a) * (A(h) * eu + 1.1 * A(up) * eg)
                                  + 2 * near * A(a * h * up)).sum(axis=1)
        np.add.at(err["dx"], t, edg @ A(m1) + edu @ A(m3) + dot(2 * I) * (A(dg) @ A(m1) + A(du) @ A(m3)))
        n = dot(len(t))
        err["dw1"][e] = edg.T @ A(xe) + n * (A(dg).T @ A(xe))
        err["dw3"][e] = edu.T @ A(xe) + n * (A(du).T @ A(xe))
        err["dw2"][e] = A(de).T @ eact + n * (A(de).T @ A(act))
    if errors is not None:
        out |= {"e_" + k: v for k, v in err.items()}
    return out
