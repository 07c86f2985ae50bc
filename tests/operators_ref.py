"""Plain 64-bit forms of the handle-less operators and the tolerances of their kernels.

A tolerance counts roundings: H(t) = finfo(t).eps / 2 is half a step of the output's type,
E = 2^-24 half a step of fp32.  A sum of n fp32 terms whose longest chain of additions is c is
off by at most c E sum|term| (2 E per step where the tensor cores may truncate instead of
rounding)."""
import torch

E = 2.0 ** -24


def half(dt):
    return torch.finfo(dt).eps / 2


def bounds(counts, rows):
    """First and last row of each expert as the library reads counts: negative ones are 0, and
    rows past the buffer are cut off."""
    b = [0]
    for c in counts:
        b.append(min(rows, b[-1] + max(0, int(c))))
    return b


def grouped(op, a, b, counts):
    """(result, tolerance) in 64 bits for mm (x, w), dgrad (dy, w), wgrad (dy, x)."""
    rows = a.shape[0]
    bd = bounds(counts.tolist(), rows)
    a64, b64 = a.double(), b.double()
    res, tol = [], []
    for g in range(len(bd) - 1):
        s = slice(bd[g], bd[g + 1])
        if op == "wgrad":
            p, q, depth = a64[s].t(), b64[s], bd[g + 1] - bd[g]
        else:
            p, q = a64[s], b64[g].t() if op == "mm" else b64[g]
            depth = p.shape[1]
        r = p @ q
        res.append(r)
        tol.append((depth + 1) * 2 * E * (p.abs() @ q.abs()))
    if op == "wgrad":
        return torch.stack(res), torch.stack(tol)
    r, t = torch.cat(res), torch.cat(tol)
    return r, t + half(a.dtype) * (r.abs() + t)


# --------------------------------------------------------------------------- block norm
def norm_fwd(x, y, gate, wq, wp, beta, eps):
    x, y, gate, wq, wp = [None if t is None else t.double() for t in (x, y, gate, wq, wp)]
    sy = sr = u = None
    p = None
    r = x
    if y is not None:
        p = y
        if wq is not None:
            sy = (y.square().mean(1) + eps).rsqrt()
            p = y * sy[:, None] * wq
        if gate is not None:
            p = p * gate
        r = beta * x + p
    if wp is not None:
        sr = (r.square().mean(1) + eps).rsqrt()
        u = r * sr[:, None] * wp
    return r, u, sy, sr, p


# The row sums: at most 16 additions in a thread, 5 in the butterfly and 32 over the warps, of
# positive terms each rounded once, so a mean of squares is off by a factor within 1 +- 56 E,
# its inverse root by half of that, plus the roundings of 1/d, the fma and the root.
STAT = 32 * E


def norm_fwd_tol(x, y, gate, wq, wp, beta, eps, dt):
    r, u, sy, sr, p = norm_fwd(x, y, gate, wq, wp, beta, eps)
    t32 = torch.zeros_like(r)
    if y is not None:   # beta x is rounded into the sum; p has four products and the statistic
        t32 = E * (r.abs() + beta * x.double().abs()) + (5 * E + STAT) * p.abs()
    tr = t32 + half(dt) * (r.abs() + t32)
    tu = ts = None
    if u is not None:
        # the error of r moves the statistic by at most its largest share of the row's rms
        rel = (t32.square().mean(1).sqrt() * sr)[:, None]
        t = t32 * (sr[:, None] * wp.double().abs()) + u.abs() * (rel + STAT + 3 * E)
        tu = t + half(dt) * (u.abs() + t)
        ts = sr * (rel[:, 0] + STAT)
    return tr, tu, None if sy is None else sy * STAT, ts


def norm_bwd(fwd, y, dr, du, gate, wq, wp, beta):
    """From the forward's stored r and statistics; also the magnitudes the errors scale with."""
    r, _, sy, sr = [None if t is None else t.double() for t in fwd]
    y, dr, du, gate, wq, wp = [None if t is None else t.double() for t in (y, dr, du, gate, wq, wp)]
    g = torch.zeros_like(r) if dr is None else dr
    mag = g.abs()
    d_pre = m_pre = None
    if wp is not None:
        xh = r * sr[:, None]
        d_pre, m_pre = (du * xh).sum(0), (du * xh).abs().sum(0)
        dh = du * wp
        g = g + sr[:, None] * (dh - xh * (dh * xh).mean(1, keepdim=True))
        mag = mag + sr[:, None] * (dh.abs() + xh.abs() * (dh * xh).abs().mean(1, keepdim=True))
    out = {"dx": (beta * g, abs(beta) * mag), "d_pre": (d_pre, m_pre)}
    if y is not None:
        yh = y if sy is None else y * sy[:, None]
        q, m = g, mag
        w = 1.0 if wq is None else wq
        if gate is not None:
            ax = 0 if gate.dim() == 1 else 1
            out["d_gate"] = ((g * yh * w).sum(ax, keepdim=ax == 1), (mag * (yh * w).abs()).sum(ax, keepdim=ax == 1))
            q, m = g * gate, mag * gate.abs()
        if wq is not None:
            out["d_post"] = ((q * yh).sum(0), (m * yh.abs()).sum(0))
            q, m = q * wq, m * wq.abs()
            q, m = (sy[:, None] * (q - yh * (q * yh).mean(1, keepdim=True)),
                    sy[:, None] * (m + yh.abs() * (m * yh.abs()).mean(1, keepdim=True)))
        out["dy"] = (q, m)
    return out


# Elements of dx and dy: two row means (each a sum with a chain of at most 53 additions) and
# fewer than 20 products, all within 128 E of the terms' magnitudes.
BWD = 128 * E


def bwd_col_tol(rows):
    """A parameter's gradient: a CTA's rows in order, 592 CTAs' sums in 32 chains, then those."""
    return BWD + (rows / 592 + 1 + 592 / 32 + 1 + 32) * E


def norm_sq(ts):
    return sum(float(t.double().square().sum()) for t in ts)
