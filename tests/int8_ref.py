"""Plain 64-bit forms of the int8 operators and layer norms, with the bound that each
float32 kernel has to keep, element by element (F, u and rounded as in block_ref)."""
import torch

from block_ref import F, act_pair, epilogue, rounded, u  # noqa: F401


def codes(x):
    """(codes in 64 bits, scales float32) of rows by the definition: float32 quotients
    (a float32 quotient is the 64-bit quotient of the same numbers, rounded)."""
    v = x.double()
    amax = v.abs().amax(1)
    s = (amax / 127.0).float()
    bad = ~torch.isfinite(amax)
    safe = torch.where((s == 0) | bad, torch.ones_like(s), s).double()
    q = (v / safe[:, None]).float().double().round().clamp(-127, 127)
    q = torch.where((bad | (s == 0))[:, None], torch.zeros_like(q), q)
    return q, torch.where(bad, torch.full_like(s, float("nan")), s)


def linear(q, s, w, u_n, bias, residual, act, t):
    """y and its bound as type t. The integer sum is exact; it is rounded once to
    float32, multiplied by the token's scale (once more) and by the channel's in an fma
    with the bias (once more)."""
    acc = q @ w.double().t()
    prod = acc * s.double()[:, None] * u_n.double()
    z = prod if bias is None else prod + bias.double()
    ez = 3 * F * prod.abs() + F * z.abs()
    return epilogue(z, ez, act, None if residual is None else residual.double(), t)


def route(logits, k):
    """Picks (ties to the lower expert) and softmax weights of float32 logits, 64-bit."""
    key = torch.where(logits == 0, torch.zeros_like(logits), logits).double()   # -0 ties +0
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    w = torch.exp(top - top[:, :1])
    return ids, w / w.sum(1, keepdim=True)


def layer(logits, x, w13, s13, w2, s2, k, residual, t):
    """(ids, w, out, bound of out). A code of h may differ by one where h / hs lies
    within its float32 error of the middle between two whole numbers; every other code
    is the same."""
    T, H = x.shape
    I = w2.shape[2]
    ids, w = route(logits, k)
    q, xs = codes(x)
    out = torch.zeros((T, H), dtype=torch.float64, device=x.device)
    err = torch.zeros_like(out)
    mag = torch.zeros_like(out)
    for e in torch.unique(ids).tolist():
        tok, pick = torch.where(ids == e)
        prod = (q[tok] @ w13[e].double().t()) * xs[tok].double()[:, None] * s13[e].double()
        ez = 3 * F * prod.abs()
        g, up = prod[:, :I], prod[:, I:]
        eg, eu = ez[:, :I], ez[:, I:]
        sg = act_pair(g, "silu")[0]
        h = sg * up
        # the exponential's argument is rounded: |g| F relative to its value
        es = 1.1 * eg + (16 + g.abs()) * F * (sg.abs() + eg)
        eh = es * (up.abs() + eu) + sg.abs() * eu + 2 * F * h.abs()
        amax = h.abs().amax(1, keepdim=True)
        hs = amax / 127
        ehs = torch.where(amax > 0, eh.amax(1, keepdim=True) / amax.clamp(min=1e-300) + 2 * F, 0)
        c = torch.where(amax > 0, h / hs.clamp(min=1e-300), 0)
        ec = torch.where(amax > 0, eh / hs.clamp(min=1e-300) + c.abs() * (ehs + 2 * F), 0)
        flip = ((c - torch.floor(c) - 0.5).abs() <= ec).double()
        y = (c.round() @ w2[e].double().t()) * hs * s2[e].double()
        ey = (flip @ w2[e].double().abs().t()) * hs * s2[e].double().abs() + y.abs() * (ehs + 4 * F)
        wj = w[tok, pick][:, None]
        out.index_add_(0, tok, wj * y)
        # softmax over k picks: exponential, sum and division
        err.index_add_(0, tok, wj * ey * (1 + (k + 16) * F) + (k + 16) * F * wj * y.abs())
        mag.index_add_(0, tok, wj * y.abs())
    if residual is not None:
        out = out + residual.double()
        mag = mag + residual.double().abs()
    err = err + (k + 3) * F * mag
    return ids, w, out, rounded(out, err, t)


def _mean(v):
    return v.mean(-1, keepdim=True)


def layer_norm(r, y, w, b, eps, tr, t):
    """((r_out, bound) or None, (h, bound)). A float32 sum of H values is off by at most
    H F times the sum of their magnitudes."""
    H = r.shape[1]
    gam = (H + 8) * F
    er = torch.zeros_like(r)
    out = None
    if y is not None:
        r = r + y
        er = F * r.abs()
        out = (r, rounded(r, er, tr))
    m = _mean(r)
    em = gam * _mean(r.abs()) + _mean(er)
    c = r - m
    ec = er + em + F * c.abs()
    var = _mean(c * c)
    ev = _mean(2 * c.abs() * ec + ec * ec) + gam * var
    p = 1 / torch.sqrt(var + eps)
    rel = 0.5 * ev / (var + eps) + 4 * F
    rel = rel + 2 * rel * rel          # the root's second order
    xh = c * p
    h = xh * w
    eh = (ec * p + xh.abs() * (rel + 2 * F)) * w.abs()
    if b is not None:
        h = h + b
    eh = eh + F * h.abs()
    return out, (h, rounded(h, eh, t))


def layer_norm_backward(r, dr_out, dh, w, eps):
    """{name: (value, bound before its rounding)}"""
    T, H = r.shape
    gam = (H + 8) * F
    m = _mean(r)
    em = gam * _mean(r.abs())
    c = r - m
    ec = em + F * c.abs()
    var = _mean(c * c)
    ev = _mean(2 * c.abs() * ec + ec * ec) + gam * var
    p = 1 / torch.sqrt(var + eps)
    rel = 0.5 * ev / (var + eps) + 4 * F
    rel = rel + 2 * rel * rel
    xh = c * p
    ex = ec * p + xh.abs() * (rel + F)
    d = dh * w
    ed = F * d.abs()
    md, emd = _mean(d), gam * _mean(d.abs()) + _mean(ed)
    mx = _mean(d * xh)
    emx = _mean(d.abs() * ex + ed * xh.abs()) + (gam + 2 * F) * _mean((d * xh).abs())
    inner = d - md - xh * mx
    mag = d.abs() + md.abs() + (xh * mx).abs()
    ei = ed + emd + ex * mx.abs() + xh.abs() * emx + 4 * F * mag
    dr = p * inner
    edr = p * ei + (rel + 2 * F) * p * (inner.abs() + ei)
    if dr_out is not None:
        dr = dr + dr_out
        edr = edr + F * (dr.abs() + dr_out.abs())
    each = dh * xh
    sums = (T + 4) * F
    return {"dr": (dr, edr + F * dr.abs()),
            "dw": (each.sum(0), (dh.abs() * ex).sum(0) + sums * each.abs().sum(0)),
            "db": (dh.sum(0), sums * dh.abs().sum(0))}
