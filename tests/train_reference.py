"""Plain 64-bit forms of what training a draft uses beside the packed
attention core, written out from their definitions (test infrastructure)."""
import numpy as np
import torch


def frequencies(theta, d):
    return torch.from_numpy(np.float32(np.power(float(theta), -2.0 * np.arange(d // 2) / d))
                            .astype(np.float64))


def turn(x, angle, back=False):
    """Pairs (j, j + d/2) of x [..., heads, d] turned by angle [..., d/2]."""
    c, s = torch.cos(angle).unsqueeze(-2), torch.sin(angle).unsqueeze(-2)
    if back:
        s = -s
    a, b = x.chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def qk_rope(x, gain, positions, theta, eps):
    """x [B, R, heads, d] float64 -> (y, its size before the rotation's
    cancellation: |z_j| + |z_{j+d/2}| of each pair)."""
    d = x.shape[-1]
    z = gain * x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    angle = positions.double().unsqueeze(-1) * frequencies(theta, d)
    a, b = z.abs().chunk(2, -1)
    return turn(z, angle), torch.cat([a + b, a + b], -1)


def qk_rope_backward(x, gain, positions, theta, eps, d_y):
    """(dx, dgain) and the sizes of the terms that their errors follow."""
    d = x.shape[-1]
    angle = positions.double().unsqueeze(-1) * frequencies(theta, d)
    w = turn(d_y, angle, back=True)
    a, b = d_y.abs().chunk(2, -1)
    w_size = torch.cat([a + b, a + b], -1)
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    u = w * gain
    dx = r * (u - x * r * r * (u * x).mean(-1, keepdim=True))
    size = r * (w_size * gain.abs() +
                x.abs() * r * r * (w_size * gain.abs() * x.abs()).mean(-1, keepdim=True))
    dg = (w * x * r).sum((0, 1, 2))
    return dx, dg, size, (w_size * x.abs() * r).sum((0, 1, 2))


def linear_cross_entropy(x, w, target, d_nll):
    """nll, lse of every row and the gradients of sum(d_nll * nll) in x and w;
    a target outside the vocabulary: no loss, no gradient."""
    N, V = x.shape[0], w.shape[0]
    held = (target >= 0) & (target < V)
    nll, lse = torch.zeros(N).double(), torch.zeros(N).double()
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    at = torch.nonzero(held).flatten()
    if len(at):
        t = target[at].long()
        z = x[at] @ w.t()
        lse[at] = torch.logsumexp(z, 1)
        one = torch.arange(len(at))
        nll[at] = lse[at] - z[one, t]
        g = torch.exp(z - lse[at][:, None])
        g[one, t] -= 1.0
        g = g * d_nll[at][:, None]
        dx[at] = g @ w
        dw = g.t() @ x[at]
    return nll, lse, dx, dw
