"""Plain float64 forms of the layers between convolutions, written from their
definitions with torch on the CPU (loops over segments, dense products)."""

import numpy as np
import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
EPS32 = 2.0 ** -24


def segments(ids, count):
    """(seg, order) of integer keys: a stable sort, keys outside [0, count) last."""
    key = np.where((ids < 0) | (ids >= count), count, ids)
    order = np.argsort(key, kind="stable")
    seg = np.array([(key < s).sum() for s in range(count + 1)])
    return seg.astype(np.int32), order.astype(np.int32)


def positions(seg, order, s):
    r = np.arange(seg[s], seg[s + 1])
    return torch.from_numpy(r if order is None else order[r].astype(np.int64))


def act(z, kind):
    if kind == "relu":
        return torch.clamp(z, min=0)
    return z * torch.sigmoid(z) if kind == "silu" else z


def slope(z, kind):
    if kind == "relu":
        return (z > 0).double()
    if kind == "silu":
        sig = torch.sigmoid(z)
        return sig + z * sig * (1 - sig)
    return torch.ones_like(z)


def norm_fwd(x, gamma, beta, seg, order, groups, eps, kind):
    """y, mean, rstd, and z (before the activation) in float64."""
    x = x.double()
    n, c = x.shape
    S = len(seg) - 1
    y, z_all = torch.zeros_like(x), torch.zeros_like(x)
    mean, rstd = torch.zeros(S, groups, dtype=torch.float64), torch.full((S, groups), eps, dtype=torch.float64) ** -0.5
    for s in range(S):
        at = positions(seg, order, s)
        if len(at) == 0:
            continue
        v = x[at].view(len(at), groups, -1)
        mean[s] = v.mean((0, 2))
        rstd[s] = (((v - mean[s][:, None]) ** 2).mean((0, 2)) + eps) ** -0.5
        xh = ((v - mean[s][:, None]) * rstd[s][:, None]).reshape(len(at), c)
        z = xh * (1.0 if gamma is None else gamma.double()) + (0.0 if beta is None else beta.double())
        z_all[at] = z
        y[at] = act(z, kind)
    return y, mean, rstd, z_all


def norm_bwd(dy, x, gamma, beta, mean, rstd, seg, order, groups, kind):
    """dx, dgamma, dbeta in float64 from the given statistics, by the formula."""
    x, dy, mean, rstd = x.double(), dy.double(), mean.double(), rstd.double()
    n, c = x.shape
    ga = torch.ones(c, dtype=torch.float64) if gamma is None else gamma.double()
    be = torch.zeros(c, dtype=torch.float64) if beta is None else beta.double()
    dx, dgamma, dbeta = torch.zeros_like(x), torch.zeros_like(ga), torch.zeros_like(ga)
    for s in range(len(seg) - 1):
        at = positions(seg, order, s)
        if len(at) == 0:
            continue
        k = len(at)
        xh = ((x[at].view(k, groups, -1) - mean[s][:, None]) * rstd[s][:, None]).reshape(k, c)
        dz = dy[at] * slope(xh * ga + be, kind)
        dgamma += (dz * xh).sum(0)
        dbeta += dz.sum(0)
        u, w = (dz * ga).view(k, groups, -1), xh.view(k, groups, -1)
        d = u - u.mean((0, 2))[:, None] - w * (u * w).mean((0, 2))[:, None]
        dx[at] = (d * rstd[s][:, None]).reshape(k, c)
    return dx, dgamma, dbeta


def philox(counter, key):
    """Philox4x32-10 on Python integers: four 32-bit words of one block."""
    c, k, w = list(counter), list(key), 0xFFFFFFFF
    for _ in range(10):
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(q >> 32) ^ c[1] ^ k[0], q & w, (p >> 32) ^ c[3] ^ k[1], p & w]
        k = [(k[0] + 0x9E3779B9) & w, (k[1] + 0xBB67AE85) & w]
    return c


def dropout_words(seed, offset, first, count):
    """Words of the elements first .. first + count - 1."""
    w = 0xFFFFFFFF
    out = []
    for b in range(first // 4, (first + count - 1) // 4 + 1):
        out += philox((b & w, b >> 32, offset & w, offset >> 32), (seed & w, seed >> 32))
    skip = first % 4
    return np.array(out[skip:skip + count], dtype=np.uint64)


def grouped_fwd(x, w, seg, x_rows, y_rows, m):
    """y and the sums of absolute products, float64."""
    x, w = x.double(), w.double()
    y, mag = torch.zeros(m, w.shape[2], dtype=torch.float64), torch.zeros(m, w.shape[2], dtype=torch.float64)
    for g in range(w.shape[0]):
        a, b = positions(seg, x_rows, g), positions(seg, y_rows, g)
        y[b] = x[a] @ w[g]
        mag[b] = x[a].abs() @ w[g].abs()
    return y, mag


def grouped_wgrad(x, dy, seg, x_rows, y_rows):
    """dW and the sums of absolute products, float64."""
    x, dy = x.double(), dy.double()
    S = len(seg) - 1
    dw = torch.zeros(S, x.shape[1], dy.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(dw)
    for g in range(S):
        a, b = positions(seg, x_rows, g), positions(seg, y_rows, g)
        dw[g] = x[a].T @ dy[b]
        mag[g] = x[a].T.abs() @ dy[b].abs()
    return dw, mag
