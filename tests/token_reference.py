"""Plain float64 forms (CPU, dense) of the token operators with, beside each
result, an elementwise bound of the error that an implementation may make which

* rounds results, softmax weights, score gradients and gz to the 16-bit type
  (relative u = 2^-8 for bfloat16, 2^-11 for float16; float16 also loses up to
  2^-25 absolutely among its subnormals), once each, and
* accumulates in 32 bits: scores off by at most about 1e-4 relative in their
  exponential (products of a hundred terms, distances of a few hundred times
  a slope), sums and products off by 1e-5 of the sum of magnitudes.

The bounds are first-order sums of those roundings through the formulas.
"""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
FLOOR = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
E = 1e-4     # relative, of exp(score) held in 32 bits
E32 = 1e-5   # of a sum of magnitudes accumulated in 32 bits


def d(t):
    return None if t is None else t.detach().cpu().double()


def within(got, ref, bound, what=""):
    got = d(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    off = (got - ref).abs()
    ok = (off <= bound) | (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    if not bool(ok.all()):
        worst = torch.where(ok, torch.zeros_like(off), off / bound.clamp_min(1e-300)).nan_to_num(float("inf"))
        at = int(worst.argmax())
        raise AssertionError("%s: %d of %d outside; worst at %d: %r for %r, bound %r" % (
            what, int((~ok).sum()), ok.numel(), at, float(got.flatten()[at]), float(ref.flatten()[at]),
            float(bound.flatten()[at])))


# ------------------------------------------------------------------ rotary
def rope(x, pos, freq, sections, interleaved, sign=1.0):
    """(result, bound): the angle's product carries its rounding error along, so
    sine and cosine are within a few 2^-24 and products add as many again."""
    dtype = x.dtype
    x, pos, freq = d(x), d(pos), d(freq)
    pos = pos if pos.dim() == 3 else pos[None]
    R = sum(sections)
    out, mag = x.clone(), torch.zeros_like(x)
    k = 0
    for a, n in enumerate(sections):
        for _ in range(n):
            t = sign * (pos[..., a] * freq[k])[..., None]
            i, j = (2 * k, 2 * k + 1) if interleaved else (k, k + R)
            out[..., i] = x[..., i] * t.cos() - x[..., j] * t.sin()
            out[..., j] = x[..., j] * t.cos() + x[..., i] * t.sin()
            mag[..., i] = mag[..., j] = x[..., i].abs() + x[..., j].abs()
            k += 1
    return out, U[dtype] * out.abs() + 2.0 ** -21 * mag + FLOOR[dtype]


# --------------------------------------------------------------- attention
def visible(B, Sq, Sk, causal=False, prefix=None, doc_q=None, doc_k=None):
    v = torch.ones((B, Sq, Sk), dtype=torch.bool)
    if causal:
        i, j = torch.arange(Sq)[:, None], torch.arange(Sk)[None]
        c = (j <= i + Sk - Sq)[None].expand(B, Sq, Sk)
        if prefix is not None:
            c = c | (j[None] < prefix.cpu()[:, None, None])
        v = v & c
    if doc_q is not None:
        dq, dk = ((t.cpu() if t.dim() == 2 else t.cpu()[None].expand(B, -1)) for t in (doc_q, doc_k))
        v = v & (dq[:, :, None] == dk[:, None, :]) & (dq >= 0)[:, :, None]
    return v


def attention(q, k, v, scale, cap=0.0, pos_q=None, pos_k=None, slopes=None, go=None, **mask):
    """Dict of (result, bound) pairs: o, lse and, with go, gq, gk, gv."""
    dtype = q.dtype
    u, fl = U[dtype], FLOOR[dtype]
    q, k, v, go, pos_q, pos_k, slopes = (d(t) for t in (q, k, v, go, pos_q, pos_k, slopes))
    B, Sq, Hq, D = q.shape
    Sk, Hk = k.shape[1:3]
    G = Hq // Hk
    vis = visible(B, Sq, Sk, **mask)[:, None]                     # B 1 Sq Sk
    # what is masked for everyone has no effect, whatever it holds
    kk = k.masked_fill(~vis.any(2)[:, 0, :, None, None], 0.0) if Sq else k
    vv = v.masked_fill(~vis.any(2)[:, 0, :, None, None], 0.0) if Sq else v
    K, V = (t.repeat_interleave(G, 2).permute(0, 2, 1, 3) for t in (kk, vv))
    Q = q.permute(0, 2, 1, 3)
    s = scale * (Q @ K.transpose(2, 3))
    slope = torch.ones_like(s)
    if cap:
        t = torch.tanh(s / cap)
        s, slope = cap * t, 1 - t * t
    if slopes is not None:
        pq, pk = (p if p.dim() == 3 else p[None] for p in (pos_q, pos_k))
        far = (pq[:, :, None] - pk[:, None]).abs()                # b Sq Sk A
        s = s - torch.einsum("ha,bija->bhij", slopes, far.expand(B, -1, -1, -1))
    s = s.masked_fill(~vis, -math.inf)
    seen = vis.any(-1, keepdim=True)
    lse = torch.logsumexp(s, -1, keepdim=True) if Sk else torch.full((B, Hq, Sq, 1), -math.inf, dtype=torch.float64)
    lse = lse.masked_fill(~seen, -math.inf)
    p = torch.exp(s - lse.masked_fill(~seen, 0.0)).masked_fill(~vis, 0.0)
    top = s.amax(-1, keepdim=True).masked_fill(~seen, 0.0) if Sk else torch.zeros_like(lse)
    few = fl * torch.exp(top - lse.masked_fill(~seen, 0.0)) * vis  # weights are rounded relative to the row's largest
    o = p @ V
    eo = u * o.abs() + ((u + E) * p + few) @ V.abs() + fl
    back = lambda t: t.permute(0, 2, 1, 3)  # noqa: E731
    out = {"o": (back(o), back(eo)), "lse": (lse[..., 0], torch.full_like(lse[..., 0], E) + 2.0 ** -22 * lse[..., 0].abs().nan_to_num(0, 0, 0))}
    if go is None:
        return out
    g = go.permute(0, 2, 1, 3)
    gg = g.masked_fill(~seen, 0.0)
    QQ = Q.masked_fill(~seen, 0.0)
    dp, mag = gg @ V.transpose(2, 3), gg.abs() @ V.abs().transpose(2, 3)
    delta = (gg * o).sum(-1, keepdim=True)
    edelta = (gg.abs() * eo).sum(-1, keepdim=True)
    ds = p * (dp - delta) * slope
    eds = (u + E) * ds.abs() + p * slope * (edelta + E * (mag + delta.abs())) + fl * vis
    fold = lambda t: back(t.reshape(B, Hk, G, Sk, D).sum(2))  # noqa: E731
    gq = scale * ds @ K
    gk, gv = scale * ds.transpose(2, 3) @ QQ, p.transpose(2, 3) @ gg
    out["gq"] = back(gq), back(u * gq.abs() + abs(scale) * (eds @ K.abs())) + fl
    ek = abs(scale) * (eds.transpose(2, 3) @ QQ.abs())
    ev = ((u + E) * p + fl * vis).transpose(2, 3) @ gg.abs()
    gk, gv, ek, ev = (fold(t) for t in (gk, gv, ek, ev))
    out["gk"], out["gv"] = (gk, u * gk.abs() + ek + fl), (gv, u * gv.abs() + ev + fl)
    return out


# ------------------------------------------------------------------ linear
def act(name, z):
    if name == "relu":
        return z.clamp_min(0.0), (z > 0).double()
    if name == "gelu":
        c = torch.special.ndtr(z)
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        c = torch.sigmoid(z)
        return z * c, c * (1 + z * (1 - c))
    return z, torch.ones_like(z)


def linear(x, w, b=None, r=None, name="none"):
    dtype = x.dtype
    u, fl = U[dtype], FLOOR[dtype]
    x, w, b, r = (d(t) for t in (x, w, b, r))
    z, mag = x @ w.T, x.abs() @ w.abs().T
    if b is not None:
        z, mag = z + b, mag + b.abs()
    y, _ = act(name, z)
    ey = 1.2 * E32 * mag + E32 * z.abs()      # |act'| <= 1.13
    if r is not None:
        y, ey = y + r, ey + E32 * r.abs()
    return {"y": (y, u * y.abs() + ey + fl), "z": (z, u * z.abs() + E32 * mag + fl)}


def linear_grads(x, w, z, gy, name="none"):
    dtype = x.dtype
    u, fl = U[dtype], FLOOR[dtype]
    x, w, z, gy = (d(t) for t in (x, w, z, gy))
    gz = gy if name == "none" else gy * act(name, z)[1]
    e = 0.0 * gz.abs() if name == "none" else u * gz.abs() + E32 * gy.abs() + fl
    gx, gw, gb = gz @ w, gz.T @ x, gz.sum(0)
    e32 = E32 * gz.abs()
    return {"gx": (gx, u * gx.abs() + (e + e32) @ w.abs() + fl), "gw": (gw, u * gw.abs() + (e + e32).T @ x.abs() + fl),
            "gb": (gb, u * gb.abs() + E32 * (gz.abs() + gy.abs()).sum(0) + fl)}
