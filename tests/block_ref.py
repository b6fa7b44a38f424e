"""Plain 64-bit forms of the block operators, each with the bound its float32
kernel has to keep, element by element.

Bounds: u(t) = eps(t) / 2 is half a step of the output's type; a float32 sum of n
products is off by at most (n + 2) 2^-24 times the sum of their magnitudes, in
any order. An operand that is rounded on its way adds u times its magnitude.
"""
import torch

F = 2.0 ** -24          # half a step of float32
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
SLOPE = {"none": 1.0, "relu": 1.0, "silu": 1.1, "gelu": 1.13}     # largest |act'|
CURVE = {"none": 0.0, "relu": 0.0, "silu": 0.5, "gelu": 0.8}      # largest |act''| (off the kink)


def u(t):
    return torch.finfo(t).eps / 2


def act_pair(z, act):
    """(act(z), act'(z)) element-wise in 64 bits."""
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        c = 0.5 * torch.erfc(-z * 0.5 ** 0.5)
        return z * c, c + z * torch.exp(-z * z / 2) * (2 * torch.pi) ** -0.5
    return z, torch.ones_like(z)


def act_fwd(z, act):
    if act == "swiglu":
        g, h = z.chunk(2, -1)
        return act_pair(g, "silu")[0] * h
    return act_pair(z, act)[0]


def act_bwd(dy, z, act):
    if act == "none":
        return dy
    if act == "swiglu":
        g, h = z.chunk(2, -1)
        v, d = act_pair(g, "silu")
        return torch.cat((dy * h * d, dy * v), -1)
    return dy * act_pair(z, act)[1]


def rounded(v, err, t):
    """Bound of a value with error `err` after its one rounding to t."""
    return err * (1 + u(t)) + v.abs() * u(t) + TINY[t]


def product(x, w, bias=None):
    """z = x w^T + bias and its float32 bound; x, w in 64 bits."""
    K = x.shape[1]
    z = x @ w.t()
    mag = x.abs() @ w.abs().t()
    if bias is not None:
        z = z + bias
        mag = mag + bias.abs()
    return z, (K + 3) * F * mag


def epilogue(z, ez, act, residual, t):
    """y = act(z) + residual and its bound as type t. The activations' hardware
    exponential and reciprocal are within 4 float32 steps of the exact value
    relative to their result's magnitude bound |z|."""
    if act == "swiglu":
        g, h = z.chunk(2, -1)
        eg, eh = ez.chunk(2, -1)
        s = act_pair(g, "silu")[0]
        y = s * h
        es = 1.1 * eg + 16 * F * (s.abs() + eg)
        e = es * (h.abs() + eh) + s.abs() * eh + 2 * F * y.abs()
    else:
        y = act_pair(z, act)[0]
        e = SLOPE[act] * ez + (0 if act in ("none", "relu") else 16 * F) * (z.abs() + ez)
    if residual is not None:
        e = e + F * (y.abs() + residual.abs())
        y = y + residual
    return y, rounded(y, e, t)


def dz_pair(dy, z, act, t, from_t=True):
    """dz and the bound of the dz that enters the products (rounded to t unless
    it is dy itself), and of the float32 dz (for the bias sum)."""
    dz = act_bwd(dy, z, act)
    if act == "none":
        e32 = torch.zeros_like(dz)
    elif act == "swiglu":
        g, h = z.chunk(2, -1)
        e32 = 32 * F * torch.cat((dy.abs() * h.abs() * (1 + g.abs()), dy.abs() * (1 + g.abs())), -1)
    else:
        e32 = 32 * F * dy.abs() * (1 + z.abs())
    exact = act == "none" and from_t
    return dz, (e32 if exact else rounded(dz, e32, t)), e32


def close(got, ref, bound, what):
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    g = got.double()
    assert torch.isfinite(g).all(), f"{what}: non-finite values"
    err = (g - ref).abs()
    if err.numel() == 0:
        return
    worst = (err / bound.clamp(min=1e-300)).max().item()
    assert worst <= 1.0, f"{what}: error {worst:.3g} times its bound"


# ------------------------------------------------------------------- norms --
def _sum(v):
    return v.sum(-1, keepdim=True)


def norm_forward(r, y, w_post, w_pre, gate, scale, eps, tr, t):
    """(r_out, bound), (h, bound); gate broadcastable to [T, H]."""
    H = r.shape[1]
    gam = (H + 16) * F
    er = torch.zeros_like(r)
    if y is not None:
        p = 1 / torch.sqrt(_sum(y * y) / H + eps) if w_post is not None else 1.0
        n = y * p * (w_post if w_post is not None else 1.0)
        n = scale * n * (gate if gate is not None else 1.0)
        er = gam * n.abs() + F * (r.abs() + n.abs())
        r = r + n
    out = (r, rounded(r, er, tr))
    if w_pre is None:
        return out, None
    q = 1 / torch.sqrt(_sum(r * r) / H + eps)
    h = r * q * w_pre
    # the mean square moves by at most its relative rounding and by er
    rel = gam + torch.sqrt(_sum(er * er) / _sum(r * r).clamp(min=1e-300))
    eh = er * q * w_pre.abs() + h.abs() * rel
    return out, (h, rounded(h, eh, t))


def norm_backward(r, dr_out, dh, y, w_post, w_pre, gate, scale, eps):
    """Every gradient in 64 bits with its float32 bound (before its rounding)."""
    like = r if r is not None else dr_out
    T, H = like.shape
    gam = 4 * (H + 16) * F
    out = {}
    dr = dr_out if dr_out is not None else torch.zeros_like(like)
    edr = 2 * F * dr.abs()
    if dh is not None:
        q = 1 / torch.sqrt(_sum(r * r) / H + eps)
        d = dh * w_pre
        dr = dr + q * d - r * q ** 3 * _sum(d * r) / H
        edr = edr + gam * (q * d.abs() + r.abs() * q ** 3 * _sum((d * r).abs()) / H)
        each = dh * r * q
        out["dw_pre"] = (each.sum(0), (gam + (T + 2) * F) * each.abs().sum(0))
    out["dr"] = (dr, edr + 2 * F * dr.abs())
    if y is None:
        return out
    g = gate if gate is not None else torch.ones(1, dtype=r.dtype if r is not None else dr.dtype, device=dr.device)
    w = w_post if w_post is not None else torch.ones(H, dtype=dr.dtype, device=dr.device)
    p = 1 / torch.sqrt(_sum(y * y) / H + eps) if w_post is not None else torch.ones_like(_sum(y))
    c = abs(scale)
    dn = scale * g * dr
    edn = c * g.abs() * edr + 4 * F * dn.abs()
    e, ee = dn * w, edn * w.abs() + F * (dn * w).abs()
    if w_post is not None:
        dy = p * e - y * p ** 3 * _sum(e * y) / H
        edy = (p * ee + y.abs() * p ** 3 * _sum(ee * y.abs()) / H +
               gam * (p * e.abs() + y.abs() * p ** 3 * _sum((e * y).abs()) / H))
    else:
        dy, edy = e, ee + F * e.abs()
    out["dy"] = (dy, edy)
    each = dn * y * p
    out["dw_post"] = (each.sum(0), (edn * y.abs() * p).sum(0) +
                      (gam + (T + 2) * F) * each.abs().sum(0))
    n = y * p * w
    dg = scale * dr * n
    edg = c * edr * n.abs() + gam * dg.abs()
    out["dgate_element"] = (dg, edg)
    out["dgate_channel"] = (dg.sum(0), edg.sum(0) + (T + 2) * F * dg.abs().sum(0))
    out["dgate_token"] = (_sum(dg), _sum(edg) + (H + 2) * F * _sum(dg.abs()))
    return out
