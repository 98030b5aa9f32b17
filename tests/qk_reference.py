"""RMSNorm of query and key heads with the rotation by position, and its gradient, in 64 bits."""
import torch


def _angles(positions, inv_freq, axis):
    pos = positions if positions.dim() == 2 else positions[None]
    axis = torch.tensor([0] * inv_freq.numel() if axis is None else list(axis), device=pos.device, dtype=torch.int64)
    a = pos[axis].t().double() * inv_freq.double()                        # [tokens][pairs]
    return torch.cos(a)[:, None], torch.sin(a)[:, None]


def turn(y, cos, sin, interleaved):
    """The first 2 * pairs values of [tokens][heads][dim] turned; the others as they are."""
    n = cos.shape[-1]
    y = y.clone()
    i = torch.arange(n, device=y.device) * (2 if interleaved else 1)
    j = i + (1 if interleaved else n)
    a, b = y[..., i].clone(), y[..., j].clone()
    y[..., i], y[..., j] = a * cos - b * sin, b * cos + a * sin
    return y


def _one(x, gamma, eps):
    if gamma is None:
        return torch.ones_like(x[..., :1]), x
    rstd = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return rstd, x * rstd * gamma.double()


def _split(qkv, hq, hk, dim):
    x = qkv.double()
    return (x[:, :hq * dim].reshape(x.shape[0], hq, dim), x[:, hq * dim:(hq + hk) * dim].reshape(x.shape[0], hk, dim))


def forward(qkv, hq, hk, dim, positions, inv_freq, gamma_q, gamma_k, eps, axis=None, interleaved=False):
    cos, sin = _angles(positions, inv_freq, axis)
    return tuple(turn(_one(x, g, eps)[1], cos, sin, interleaved)
                 for x, g in zip(_split(qkv, hq, hk, dim), (gamma_q, gamma_k)))


def magnitude(qkv, hq, hk, dim, positions, inv_freq, gamma_q, gamma_k, eps, axis=None, interleaved=False):
    """|a| + |b| of every value's pair after the norm (|n| past the rotation): what a rounding of an output scales with."""
    cos, sin = _angles(positions, inv_freq, axis)
    return tuple(_both(_one(x, g, eps)[1].abs(), cos, interleaved)
                 for x, g in zip(_split(qkv, hq, hk, dim), (gamma_q, gamma_k)))


def _both(v, cos, interleaved):
    n = cos.shape[-1]
    i = torch.arange(n, device=v.device) * (2 if interleaved else 1)
    j = i + (1 if interleaved else n)
    w = v.clone()
    w[..., i] = w[..., j] = v[..., i] + v[..., j]
    return w


def backward(dq, dk, qkv, positions, inv_freq, gamma_q, gamma_k, eps, axis=None, interleaved=False):
    """dx [tokens][heads * dim], dgamma_q, dgamma_k, and what their roundings scale with (the same three)."""
    cos, sin = _angles(positions, inv_freq, axis)
    hq, hk, dim = dq.shape[1], dk.shape[1], dq.shape[2]
    xs = (None, None) if qkv is None else _split(qkv, hq, hk, dim)
    dx, dg, sx, sg = [], [], [], []
    for x, dy, g in zip(xs, (dq, dk), (gamma_q, gamma_k)):
        d = turn(dy.double(), cos, -sin, interleaved)
        size = _both(dy.double().abs(), cos, interleaved)
        if g is None:
            dx.append(d.flatten(1)), sx.append(size.flatten(1)), dg.append(None), sg.append(None)
            continue
        rstd, _ = _one(x, g, eps)
        xh, t, ts = x * rstd, d * g.double(), size * g.double().abs()
        dx.append((rstd * (t - xh * (t * xh).mean(-1, keepdim=True))).flatten(1))
        sx.append((rstd * (ts + xh.abs() * (ts * xh.abs()).mean(-1, keepdim=True))).flatten(1))
        dg.append((d * xh).sum((0, 1)))
        sg.append((size * xh.abs()).sum((0, 1)))
    return torch.cat(dx, 1), dg[0], dg[1], torch.cat(sx, 1), sg[0], sg[1]
