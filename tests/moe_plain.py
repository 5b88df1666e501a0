"""Plain 64-bit statements of the MoE-block operators (RMS norm, routing and
their backward passes, products with 4-bit weights), for the tests: numpy,
straight from the formulas in include/nvfp4.h, sharing nothing with the
library."""
import numpy as np
import torch

U = 2.0 ** -24          # half a binary32 step, relative
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
LOWEST = -3.4028234663852886e38


def host(t):
    """A device tensor's values as float64."""
    return t.detach().double().cpu().numpy()


# ---------------------------------------------------------------- norm
def rmsnorm(h, weight, eps):
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return rstd, h * rstd[:, None] * weight


def rmsnorm_backward(dy, h, rstd, weight, dh):
    g, xhat = dy * weight, h * rstd[:, None]
    dx = rstd[:, None] * (g - xhat * (g * xhat).mean(axis=1, keepdims=True))
    return dx + (0.0 if dh is None else dh), (dy * xhat).sum(axis=0)


# ---------------------------------------------------------------- routing
def clean(l):
    """Logits as the operators read them."""
    l = np.where(np.isnan(l), LOWEST, l)
    return np.clip(l, LOWEST, -LOWEST)


def scores(l, sigmoid):
    l = clean(l)
    if sigmoid:
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    e = np.exp(l - l.max(axis=1, keepdims=True))
    return e / e.sum(axis=1, keepdims=True)


def log_scores(l, sigmoid):
    """log p up to a constant of the row, without underflow."""
    l = clean(l)
    return -np.logaddexp(0.0, -l) if sigmoid else l


def route(l, k, bias=None, sigmoid=False, groups=1, top_groups=1, top2=True, renorm=True):
    T, E = l.shape
    p = scores(l, sigmoid)
    # without a bias, scores order as the logits do (also where they underflow)
    s = clean(l) if bias is None else clean(p + bias)
    ids = np.empty((T, k), dtype=np.int64)
    n = E // groups
    for t in range(T):
        keys = s[t].copy()
        if top_groups < groups:
            by = []
            for g in range(groups):
                best = np.sort((p[t] if bias is None else s[t])[g * n:(g + 1) * n])[::-1]
                if not top2:
                    best = np.sort(s[t][g * n:(g + 1) * n])[::-1]
                by.append(best[0] + best[1] if top2 and n > 1 else best[0])
            keep = sorted(range(groups), key=lambda g: (-by[g], g))[:top_groups]
            for g in range(groups):
                if g not in keep:
                    keys[g * n:(g + 1) * n] = -np.inf
        ids[t] = sorted(range(E), key=lambda e: (-keys[e], e))[:k]
    w = np.take_along_axis(p, ids, axis=1)
    if renorm:
        lw = np.take_along_axis(log_scores(l, sigmoid), ids, axis=1)
        w = np.exp(lw - lw.max(axis=1, keepdims=True))
        w = w / w.sum(axis=1, keepdims=True)
    return ids, w


def plan(ids, experts):
    flat = ids.reshape(-1)
    order = np.argsort(flat, kind="stable")
    position = np.empty_like(order)
    position[order] = np.arange(order.size)
    return np.searchsorted(flat[order], np.arange(experts + 1)), order, position


def route_backward(dw, l, ids, sigmoid, renorm, ds):
    """Softmax: dl = p (ds - sum p ds) and, for the chosen, w (dw - sum dw w)
    when renormalised (whose terms of the softmax's sum cancel exactly) or
    p dw - p sum p dw; sigmoid: (1 - p) times p ds and the chosen term."""
    p = scores(l, sigmoid)
    w = np.take_along_axis(p, ids, axis=1)
    chosen = np.zeros_like(p)
    if renorm:
        w = w / w.sum(axis=1, keepdims=True)
        term, common = w * (dw - (dw * w).sum(axis=1, keepdims=True)), 0.0
    else:
        term, common = w * dw, (w * dw).sum(axis=1, keepdims=True)
    for t in range(l.shape[0]):
        for j in range(ids.shape[1]):
            chosen[t, ids[t, j]] += term[t, j]
    if ds is None:
        ds = np.zeros_like(p)
    if sigmoid:
        return (1.0 - p) * (p * ds + chosen)
    return p * (ds - (p * ds).sum(axis=1, keepdims=True) - common) + chosen


# ---------------------------------------------------------------- products with 4-bit weights
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6])


def e2m1(codes):
    """Values of packed E2M1 codes (rows x cols/2 bytes, low nibble first)."""
    c = codes.cpu().numpy()
    return np.stack((E2M1[c & 15], E2M1[c >> 4]), axis=2).reshape(c.shape[0], -1)


def e4m3(b):
    b = b.cpu().numpy().astype(np.int64)
    e, m = b >> 3, b & 7
    return np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)


def nvfp4_weight(w, experts=1):
    """The values of an NVFP4Tensor (a stack of `experts` matrices)."""
    s = e4m3(w.scales)
    s = np.repeat(s, 16, axis=1)
    s = np.repeat(s, 16, axis=0) if w.scale_mode == 1 else s
    ts = host(w.tensor_scale)
    return e2m1(w.codes) * s * np.repeat(ts, w.rows // experts)[:, None]


def mx_weight(w):
    s = 2.0 ** (w.scales.cpu().numpy().astype(np.int64) - 127.0)
    return e2m1(w.codes) * np.repeat(s, 32, axis=1)


def swiglu(z, wabs):
    """gate sigmoid(gate) up of z = [gate, up], and how far it moves when each
    of z does by `wabs`."""
    f = z.shape[1] // 2
    g, u, dg, du = z[:, :f], z[:, f:], wabs[:, :f], wabs[:, f:]
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    return g * s * u, np.abs(s * (1.0 + g * (1.0 - s)) * u) * dg + np.abs(g * s) * du
