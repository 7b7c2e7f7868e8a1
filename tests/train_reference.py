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
    return linear_cross_entropy_sizes(x, w, target, d_nll)[:4]


def linear_cross_entropy_sizes(x, w, target, d_nll):
    """The same, and what its errors follow: the largest sum |x||w| and |z| of
    a row, and the sums of the gradients' terms without their signs."""
    N, V = x.shape[0], w.shape[0]
    held = (target >= 0) & (target < V)
    zero = lambda *s: torch.zeros(*s, dtype=x.dtype, device=x.device)  # noqa: E731
    nll, lse, z_size, z_top = zero(N), zero(N), zero(N), zero(N)
    dx, dw, dx_size, dw_size = (torch.zeros_like(t) for t in (x, w, x, w))
    at = torch.nonzero(held).flatten()
    if len(at):
        t = target[at].long()
        xa, d = x[at], d_nll[at][:, None]
        z = xa @ w.t()
        lse[at] = torch.logsumexp(z, 1)
        one = torch.arange(len(at), device=x.device)
        nll[at] = lse[at] - z[one, t]
        z_size[at] = (xa.abs() @ w.abs().t()).amax(1)
        z_top[at] = z.abs().amax(1)
        g = torch.exp(z - lse[at][:, None])
        g[one, t] = 0.0
        g[one, t] = -g.sum(1)  # p_t - 1, without cancelling
        g = g * d
        dx[at] = g @ w
        dw = g.t() @ xa
        dx_size[at] = g.abs() @ w.abs()
        dw_size = g.abs().t() @ xa.abs()
    return nll, lse, dx, dw, z_size, z_top, dx_size, dw_size
