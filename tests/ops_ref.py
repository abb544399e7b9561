"""The operators of ttt_ops.h in 64 bits, and bounds of the kernels' errors.

Each reference returns, beside its results, how far a kernel that works in 32 bits may be
from them: first-order error propagation through the same formulas.  E32 = 2^-24 is half a
step of fp32; results are then rounded once to the output's type, half a step of it
(`half_step`: bf16 2^-8, fp32 2^-24) relative to the value.
"""
import math

import torch

E32 = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounded(value, err, dtype):
    """The bound of `value` (known to `err`) after its rounding to `dtype`: one rounding, which is
    exact to half a step of the value or, below the normal range, to half the smallest step."""
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    return err + half_step(dtype) * (value.abs() + err) + tiny


def check(name, got, want, bound):
    got = got.double().cpu()
    want, bound = want.cpu(), bound.cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    off = (got - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        i = torch.nonzero(bad)[0].tolist()
        at = tuple(i)
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} values off, first at {i}: got "
                             f"{got[at].item()}, want {want[at].item()}, bound {bound[at].item():.3g}")


# ------------------------------------------------------------------------- rope
def rope(x, pos, pairs, base, pairing, inverse=False):
    """x [B,H,N,d] (64 bits), pos [N,A] or [B,N,A]; returns y and its error bound before rounding.

    Error: the angle is reduced in 64 bits to |turn| <= 1/2 and rounded to 32 (2^-26 turns, 2^-23.3
    radians); sine and cosine are taken to 2^-21.1 absolute at worst (the hardware's approximation on
    [-pi, pi], used for bf16), the argument's product with 2 pi adds 2^-22.3; the two products and
    their sum 3 half steps of 32 bits.  In all below (|x_p| + |x_q|) 2^-20."""
    base = list(base) if isinstance(base, (list, tuple)) else [base] * len(pairs)
    pos = pos.double()
    pos = pos if pos.dim() == 3 else pos[None].expand(x.shape[0], -1, -1)
    m = sum(pairs)
    y, err = x.clone(), torch.zeros_like(x)
    i = 0
    for a, n in enumerate(pairs):
        for j in range(n):
            phi = pos[:, None, :, a] * base[a] ** (-j / n)
            c, s = torch.cos(phi), torch.sin(phi) * (-1 if inverse else 1)
            p, q = (i, i + m) if pairing == "halves" else (2 * i, 2 * i + 1)
            y[..., p] = x[..., p] * c - x[..., q] * s
            y[..., q] = x[..., q] * c + x[..., p] * s
            err[..., p] = err[..., q] = (x[..., p].abs() + x[..., q].abs()) * 2.0 ** -20
            i += 1
    return y, err


# ------------------------------------------------------------------------- scan
# half steps of 32 bits that one step of the recurrence is off by, relative to |a h| + |u|: the gate
# (an exponential of at most 2 steps, a sum and a quotient: 6), its product into a running product
# (1) or a state (1), the input's product (1), the sums where partial results are joined (3)
STEP = 12 * E32


def gate(g, kind):
    a = g if kind == "value" else torch.exp(g) if kind == "exp" else torch.sigmoid(g)
    rest = 1 - g if kind == "value" else -torch.expm1(g) if kind == "exp" else torch.sigmoid(-g)
    slope = torch.ones_like(g) if kind == "value" else a if kind == "exp" else a * rest
    return a, rest, slope


def scan(g, x, kind, inp, h0=None, lengths=None, dh=None, dh_last=None):
    """Results (name -> value, bound before rounding); rows behind a sequence's end hold NaN (not compared)."""
    B, L, D = x.shape
    n = [L] * B if lengths is None else [min(max(int(v), 0), L) for v in lengths]
    zero = x.new_zeros(D)
    nan = lambda: torch.full((B, L, D), math.nan, dtype=torch.float64)  # noqa: E731
    a, rest, slope = gate(g, kind)
    u = rest * x if inp == "complement" else x
    out = {"h": nan(), "h_last": torch.zeros(B, D, dtype=torch.float64)}
    eh = {"h": nan(), "h_last": torch.zeros(B, D, dtype=torch.float64)}
    if dh is not None:
        for k in ("dg", "dx"):
            out[k], eh[k] = nan(), nan()
        out["dh0"], eh["dh0"] = torch.zeros(B, D, dtype=torch.float64), torch.zeros(B, D, dtype=torch.float64)
    for b in range(B):
        h = h0[b] if h0 is not None else zero
        size, err = h.abs(), zero.clone()
        before = []
        for t in range(n[b]):
            before.append((h, err))
            h = a[b, t] * h + u[b, t]
            step = a[b, t].abs() * size + u[b, t].abs()
            err = a[b, t].abs() * err + STEP * step
            size = step
            out["h"][b, t], eh["h"][b, t] = h, err
        out["h_last"][b], eh["h_last"][b] = h, err
        if dh is None:
            continue
        mu = dh_last[b] if dh_last is not None else zero
        size, err = mu.abs(), zero.clone()
        for t in range(n[b] - 1, -1, -1):
            lam, elam, slam = dh[b, t] + mu, err + E32 * (dh[b, t].abs() + size), dh[b, t].abs() + size
            hp, ehp = before[t]
            d = hp - x[b, t] if inp == "complement" else hp
            sd = hp.abs() + x[b, t].abs() if inp == "complement" else hp.abs()
            r = rest[b, t] if inp == "complement" else torch.ones(D, dtype=torch.float64)
            out["dx"][b, t], eh["dx"][b, t] = r * lam, r.abs() * elam + STEP * (r * lam).abs()
            s = slope[b, t]
            out["dg"][b, t] = lam * d * s
            # first order in each factor; the gate's slope and three products
            eh["dg"][b, t] = s.abs() * ((elam * (d.abs() + ehp)) + lam.abs() * (ehp + E32 * sd)) + \
                2 * STEP * (lam * d * s).abs()
            mu = a[b, t] * lam
            err = a[b, t].abs() * elam + STEP * (a[b, t].abs() * slam)
            size = a[b, t].abs() * slam
        out["dh0"][b], eh["dh0"][b] = mu, err
    return out, eh


# ------------------------------------------------------------------------- norm
# Sums run in 32 bits over at most this many additions one after the other (the rest is added
# pairwise), so a sum is off by CHAIN half steps of the sum of magnitudes at most.
CHAIN = 256 * E32


def act(z, kind):
    return z if kind == "none" else z * torch.sigmoid(z) if kind == "silu" else 0.5 * z * torch.erfc(-z / math.sqrt(2))


def act_grad(z, kind):
    if kind == "none":
        return torch.ones_like(z)
    if kind == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def norm(x, G, weight, bias, kind, eps, dy=None):
    """x [B,N,C] in 64 bits.  Results (name -> value, bound before rounding)."""
    B, N, C = x.shape
    n = C // G
    w = weight if weight is not None else x.new_ones(C)
    o = bias if bias is not None else x.new_zeros(C)
    v = x.view(B, N, G, n)
    mean = v.mean((1, 3), keepdim=True)
    var = (v - mean).square().mean((1, 3), keepdim=True)
    rstd = (var + eps).rsqrt()
    xhat = (v - mean) * rstd
    # the mean is off by CHAIN of the mean magnitude; the variance, taken about it, by CHAIN of
    # itself and the square of that; 1/sqrt by half of it and two steps
    emean = CHAIN * v.abs().mean((1, 3), keepdim=True)
    erstd = 0.5 * (CHAIN * var + emean.square()) / (var + eps) + 4 * E32
    exhat = rstd * (emean + 2 * E32 * (v.abs() + mean.abs())) + xhat.abs() * (erstd + 2 * E32)
    flat = lambda t: t.reshape(B, N, C)  # noqa: E731
    xh, exh = flat(xhat), flat(exhat)
    z = xh * w + o
    ez = w.abs() * exh + 2 * E32 * ((xh * w).abs() + o.abs())
    # |act'| <= 1.13; the activation itself: an exponential or erfc of a few steps, 8 in all, relative
    # to |z| times a factor of at most one
    out, err = {"y": act(z, kind)}, {"y": 1.13 * ez + 8 * E32 * z.abs()}
    out["mean"], err["mean"] = mean[:, 0, :, 0], (emean + E32 * mean.abs())[:, 0, :, 0]
    out["rstd"], err["rstd"] = rstd[:, 0, :, 0], (rstd * erstd)[:, 0, :, 0]
    if dy is None:
        return out, err
    dz = dy * act_grad(z, kind)
    # |act''| <= 0.8; act' is made of factors of at most 1.13 + |z| phi: 16 half steps
    edz = dy.abs() * (0.8 * ez + 16 * E32 * 1.2) + E32 * dz.abs()
    out["dbias"], err["dbias"] = dz.sum((0, 1)), (edz + CHAIN * dz.abs()).sum((0, 1))
    p = dz * xh
    ep = edz * xh.abs() + dz.abs() * exh + E32 * p.abs()
    out["dweight"], err["dweight"] = p.sum((0, 1)), (ep + CHAIN * p.abs()).sum((0, 1))
    by = lambda t: t.reshape(B, N, G, n)  # noqa: E731
    q, eq = by(dz * w), by((edz + E32 * dz.abs()) * w.abs())
    m0, em0 = q.mean((1, 3), keepdim=True), (eq + CHAIN * q.abs()).mean((1, 3), keepdim=True)
    qx, eqx = q * xhat, eq * xhat.abs() + q.abs() * exhat
    m1, em1 = qx.mean((1, 3), keepdim=True), (eqx + CHAIN * qx.abs()).mean((1, 3), keepdim=True)
    dx = rstd * (q - m0 - xhat * m1)
    size = rstd * (q.abs() + m0.abs() + (xhat * m1).abs())
    edx = rstd * (eq + em0 + exhat * m1.abs() + xhat.abs() * em1) + size * (erstd + 4 * E32)
    out["dx"], err["dx"] = flat(dx), flat(edx)
    return out, err
