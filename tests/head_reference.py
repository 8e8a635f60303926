"""Plain fp64 forms of the embedding-head operators, for the tests."""
import math

import torch


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(
            2 * math.pi)
    if act == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    return torch.ones_like(z)


def linear(X, W, b, act, R):
    z = X.double() @ W.double().t()
    if b is not None:
        z = z + b.double()
    y = _act(z, act)
    if R is not None:
        y = y + R.double()
    return y, z


def linear_backward(dY, X, W, act, Z):
    g = dY.double()
    if act != "none":
        g = g * slope(Z.double(), act)
    return g @ W.double(), g.t() @ X.double(), g.sum(0)


def layer_norm(X, gamma, beta, eps):
    x = X.double()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1 / ((c * c).mean(1) + eps).sqrt()
    y = c * rstd[:, None]
    if gamma is not None:
        y = y * gamma.double()
    if beta is not None:
        y = y + beta.double()
    return y, mean, rstd


def layer_norm_backward(dY, X, gamma, mean, rstd):
    dy, r = dY.double(), rstd.double()[:, None]
    h = (X.double() - mean.double()[:, None]) * r
    w = dy if gamma is None else dy * gamma.double()
    dx = r * (w - w.mean(1, keepdim=True) - h * (w * h).mean(1, keepdim=True))
    return dx, (dy * h).sum(0), dy.sum(0)


def _kept(labels, K):
    lab = labels.reshape(labels.shape[0], -1)
    ok = (lab >= 0) & (lab < K)
    return lab, ok, ok.any(1)


def balance_counts(labels, K):
    lab, ok, kept = _kept(labels, K)
    return torch.bincount(lab[ok].long(), minlength=K), int(kept.sum())


def balance(S, labels, counts, n, scale, coef):
    K = S.shape[1]
    lab, _, kept = _kept(labels, K)
    n = max(n, 1)
    f = counts.double() / (n * lab.shape[1])
    x = scale * S.double()
    x = torch.where(kept[:, None], x, torch.zeros_like(x))
    none = (x == -math.inf).all(1)
    x = torch.where(none[:, None], torch.zeros_like(x), x)
    p = torch.softmax(x, 1) * (kept & ~none)[:, None]
    t = (p * f).sum(1, keepdim=True)
    return coef * K / n * t.sum(), coef * scale * K / n * p * (f - t)
