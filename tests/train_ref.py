"""64-bit definitions of the training operators, with the error each result may carry.

Every function returns results in float64 beside a bound per element, counted from the
operator's own roundings: a bf16 rounding is off by at most 2^-8 of the value, f32 sums of n
products by at most n * 2^-23 of the sum of the products' magnitudes (2^-24 per addition, and
as much again for sums that truncate), the fast exponential and divide by 2^-20 of the value.
"""
import math

import torch

D = torch.float64
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
FUNC = {torch.bfloat16: 2.0 ** -20, torch.float32: 2.0 ** -21}  # activation functions, relative


def d(t):
    return None if t is None else t.to(D)


def act(z, kind):
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    if kind == "gelu":
        return z * torch.special.ndtr(z)
    return z


def act_grad(z, kind):
    if kind == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    if kind == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def linear_forward(x, w, b, r, kind):
    hs, fn, n = HALF_STEP[x.dtype], FUNC[x.dtype], x.shape[1]
    z = d(x) @ d(w).T
    mag = d(x).abs() @ d(w).abs().T
    if b is not None:
        z, mag = z + d(b), mag + d(b).abs()
    dz = (n + 2) * 2.0 ** -23 * mag
    y = act(z, kind)
    dy = 1.2 * dz + 4 * fn * (z.abs() + 1)  # |act'| <= 1.13; function error relative to |z| + 1
    if r is not None:
        y = y + d(r)
        dy = dy + 2.0 ** -23 * y.abs()
    return (y, dy + hs * (y.abs() + dy)), (z, dz + hs * (z.abs() + dz))


def linear_backward(dy, x, w, pre, kind):
    hs, fn = HALF_STEP[x.dtype], FUNC[x.dtype]
    T, N = dy.shape
    dz = d(dy)
    off = torch.zeros_like(dz)
    plain = off
    if kind != "none":
        dz = dz * act_grad(d(pre), kind)
        off = 8 * fn * d(dy).abs() * (1 + d(pre).abs())   # the derivative's own terms are <= 1 + |z|
        plain = off
        off = off + hs * (dz.abs() + off)                  # dz rounded before the products
    def prod(a, ea, b, n):
        v = a @ b
        e = ea @ b.abs() + n * 2.0 ** -23 * (a.abs() @ b.abs())
        return v, e + hs * (v.abs() + e)
    dx = prod(dz, off, d(w), N)
    dw = prod(dz.T, off.T, d(x), T)
    db = dz.sum(0)
    eb = plain.sum(0) + T * 2.0 ** -23 * dz.abs().sum(0)
    return dx, dw, (db, eb + hs * (db.abs() + eb))


def norm_forward(x, w, b, eps, kind):
    hs, H = HALF_STEP[x.dtype], x.shape[1]
    x64 = d(x)
    mu = x64.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(x64[:, :1])
    var = (x64 - mu).square().mean(-1, keepdim=True)
    rstd = (var + eps) ** -0.5
    y = (x64 - mu) * rstd * d(w)
    # the f32 mean is off by at most H 2^-24 mean|x| (summed in trees: far less), which moves
    # every element, and the variance about it by its square
    emu = (32 * 2.0 ** -24 * x64.abs().mean(-1, keepdim=True)) if kind == "layer" else 0 * mu
    ey = (emu * rstd + (64 * 2.0 ** -24 + (emu * rstd) ** 2) * ((x64 - mu) * rstd).abs()) * d(w).abs()
    if b is not None:
        y = y + d(b)
        ey = ey + 2.0 ** -23 * y.abs()
    stats = torch.cat([mu, rstd], -1)
    es = torch.cat([emu + 2.0 ** -24 * mu.abs(), rstd * (64 * 2.0 ** -24 + (emu * rstd) ** 2)], -1)
    return (y, ey + hs * (y.abs() + ey)), (stats, es)


def norm_backward(dy, x, w, stats, kind):
    hs, T = HALF_STEP[x.dtype], x.shape[0]
    mu, rstd = d(stats)[:, :1], d(stats)[:, 1:]
    xh = (d(x) - mu) * rstd
    exh = 4 * 2.0 ** -24 * (d(x).abs() + mu.abs()) * rstd
    g = d(dy) * d(w)
    b = (g * xh).mean(-1, keepdim=True)
    a = g.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(b)
    eb = 64 * 2.0 ** -24 * (g * xh).abs().mean(-1, keepdim=True) + (g.abs() * exh).mean(-1, keepdim=True)
    ea = 64 * 2.0 ** -24 * g.abs().mean(-1, keepdim=True)
    dx = rstd * (g - a - xh * b)
    ex = rstd * (ea + xh.abs() * eb + exh * b.abs() + 8 * 2.0 ** -24 * (g.abs() + a.abs() + (xh * b).abs()))
    dw = (d(dy) * xh).sum(0)
    ew = (d(dy).abs() * exh).sum(0) + (T + 4) * 2.0 ** -24 * (d(dy) * xh).abs().sum(0)
    db = d(dy).sum(0)
    edb = (T + 4) * 2.0 ** -24 * d(dy).abs().sum(0)
    return ((dx, ex + hs * (dx.abs() + ex)), (dw, ew + hs * (dw.abs() + ew)), (db, edb + hs * (db.abs() + edb)))


# ------------------------------------------------------------------ gated feed-forward
def gate_up(w, spec, e, suffix):
    if spec.gate_up_interleaved:
        p = w["gate_up" + suffix].reshape(spec.num_experts, 2 * spec.intermediate, -1)[e]
        return d(p[0::2]), d(p[1::2])
    I = spec.intermediate
    return (d(w["gate" + suffix].reshape(spec.num_experts, I, -1)[e]),
            d(w["up" + suffix].reshape(spec.num_experts, I, -1)[e]))


def gated(g, v, spec):
    """h, dh/dg, dh/dv"""
    if spec.activation == "swiglu":
        s = torch.sigmoid(g)
        return g * s * v, (s + g * s * (1 - s)) * v, g * s
    L, al = spec.swiglu_limit, spec.swiglu_alpha
    gc, vc = g.clamp(max=L), v.clamp(-L, L)
    s = torch.sigmoid(al * gc)
    return (gc * s * (vc + 1), (s + al * gc * s * (1 - s)) * (vc + 1) * (g <= L).to(D),
            gc * s * (v.abs() <= L).to(D))


def groups(spec, T, routing, dev):
    """(expert, slots, tokens, weights) of every expert with rows, in sorted order."""
    if routing is None:
        t = torch.arange(T, device=dev)
        return [(0, t, t, torch.ones(T, 1, dtype=D, device=dev))]
    off, slots, wts = routing
    o = off.tolist()
    out = []
    for e in range(spec.num_experts):
        if o[e + 1] > o[e]:
            s = slots[o[e]:o[e + 1]].long()
            out.append((e, s, s // spec.top_k, d(wts).reshape(-1)[s][:, None]))
    return out


def ffn_forward(x, w, spec, routing, residual):
    dev, dt = x.device, x.dtype
    hs, fn = HALF_STEP[dt], FUNC[dt]
    T, K, I, E = x.shape[0], spec.expert_in, spec.intermediate, spec.num_experts
    S = T * spec.top_k
    y, ey = torch.zeros(T, K, dtype=D, device=dev), torch.zeros(T, K, dtype=D, device=dev)
    pre, epre = torch.zeros(S, 2 * I, dtype=D, device=dev), torch.zeros(S, 2 * I, dtype=D, device=dev)
    p0 = 0
    for e, slots, tok, wt in groups(spec, T, routing, dev):
        wg, wu = gate_up(w, spec, e, "_w")
        wd = d(w["down_w"]).reshape(E, K, I)[e]
        u = d(x)[tok]
        g, v = u @ wg.T, u @ wu.T
        eg, ev = (u.abs() @ m.abs().T * ((K + 2) * 2.0 ** -23) for m in (wg, wu))
        bd = 0
        if spec.has_expert_bias:
            bg, bu = gate_up(w, spec, e, "_b")
            g, v = g + bg[:, 0], v + bu[:, 0]
            bd = d(w["down_b"]).reshape(E, K)[e]
        cols = (slice(0, None, 2), slice(1, None, 2)) if spec.gate_up_interleaved else (slice(0, I), slice(I, 2 * I))
        n = len(tok)
        for c, val, er in zip(cols, (g, v), (eg, ev)):
            pre[p0:p0 + n, c] = val
            epre[p0:p0 + n, c] = er + hs * (val.abs() + er)
        p0 += n
        h, hg, hv = gated(g, v, spec)
        eh = hg.abs() * eg + hv.abs() * ev + 8 * fn * (h.abs() + eg + ev)
        eh = eh + hs * (h.abs() + eh)
        o = h @ wd.T + bd
        eo = eh @ wd.abs().T + (I + 2) * 2.0 ** -23 * (h.abs() @ wd.abs().T + abs(bd))
        y.index_add_(0, tok, wt * o)
        ey.index_add_(0, tok, wt * (eo + 2.0 ** -22 * o.abs()))
    if residual is not None:
        y = y + d(residual)
        ey = ey + 2.0 ** -23 * d(residual).abs()
    return (y, ey + hs * (y.abs() + ey)), (pre, epre)


def ffn_backward(dy, x, w, pre, spec, routing):
    dev, dt = x.device, x.dtype
    hs, fn = HALF_STEP[dt], FUNC[dt]
    T, K, I, E = x.shape[0], spec.expert_in, spec.intermediate, spec.num_experts
    S = T * spec.top_k
    il, bias = spec.gate_up_interleaved, spec.has_expert_bias
    names = ["gate_up"] if il else ["gate", "up"]
    z = lambda *s: torch.zeros(*s, dtype=D, device=dev)  # noqa: E731
    val = {"x": z(T, K), "topk_w": z(S), "down_w": z(E, K, I)}
    err = {k: v.clone() for k, v in val.items()}
    for n in names:
        rows = 2 * I if il else I
        val[n + "_w"], err[n + "_w"] = z(E, rows, K), z(E, rows, K)
        if bias:
            val[n + "_b"], err[n + "_b"] = z(E, rows), z(E, rows)
    if bias:
        val["down_b"], err["down_b"] = z(E, K), z(E, K)
    p0 = 0
    for e, slots, tok, wt in groups(spec, T, routing, dev):
        n = len(tok)
        wg, wu = gate_up(w, spec, e, "_w")
        wd = d(w["down_w"]).reshape(E, K, I)[e]
        p = d(pre[p0:p0 + n])
        p0 += n
        g, v = (p[:, 0::2], p[:, 1::2]) if il else (p[:, :I], p[:, I:])
        h, hg, hv = gated(g, v, spec)
        dyt, u = d(dy)[tok], d(x)[tok]
        dh = dyt @ wd
        edh = (K + 2) * 2.0 ** -23 * (dyt.abs() @ wd.abs())
        dwt = (dh * h).sum(1)
        ewt = (edh * h.abs() + dh.abs() * 8 * fn * (h.abs() + 1e-3)).sum(1) + (I + 2) * 2.0 ** -23 * (dh * h).abs().sum(1)
        if bias:
            bd = d(w["down_b"]).reshape(E, K)[e]
            dwt = dwt + dyt @ bd
            ewt = ewt + (K + 2) * 2.0 ** -23 * (dyt.abs() @ bd.abs())
        val["topk_w"][slots] = dwt
        err["topk_w"][slots] = ewt
        scale = v.abs() + g.abs() + 1  # the derivatives' own terms
        parts = []
        for hd in (hg, hv):
            q = wt * dh * hd
            eq = wt.abs() * (edh * hd.abs() + 8 * fn * dh.abs() * (hd.abs() + scale * 2.0 ** -2))
            parts.append((q, eq + hs * (q.abs() + eq)))
        (dg, eg), (dv, ev) = parts
        val["x"].index_add_(0, tok, dg @ wg + dv @ wu)
        err["x"].index_add_(0, tok, eg @ wg.abs() + ev @ wu.abs() +
                            (2 * I + 2 + spec.top_k) * 2.0 ** -23 * (dg.abs() @ wg.abs() + dv.abs() @ wu.abs()))
        hw = wt * h
        ehw = wt.abs() * 8 * fn * (h.abs() + 1e-3)
        ehw = ehw + hs * (hw.abs() + ehw)
        val["down_w"][e] = dyt.T @ hw
        err["down_w"][e] = dyt.abs().T @ ehw + (n + 2) * 2.0 ** -23 * (dyt.abs().T @ hw.abs())
        for (q, eq), name, at in ((parts[0], "gate", slice(0, None, 2)), (parts[1], "up", slice(1, None, 2))):
            plane, rows = ("gate_up", at) if il else (name, slice(None))
            val[plane + "_w"][e, rows] = q.T @ u
            err[plane + "_w"][e, rows] = eq.T @ u.abs() + (n + 2) * 2.0 ** -23 * (q.abs().T @ u.abs())
            if bias:
                val[plane + "_b"][e, rows] = q.sum(0)
                err[plane + "_b"][e, rows] = eq.sum(0) + (n + 2) * 2.0 ** -23 * q.abs().sum(0)
        if bias:
            val["down_b"][e] = (dyt * wt).sum(0)
            err["down_b"][e] = (n + 2) * 2.0 ** -23 * (dyt * wt).abs().sum(0)
    out = {}
    for k, v in val.items():
        last = 2.0 ** -24 if k == "topk_w" else hs
        out[k] = (v, err[k] + last * (v.abs() + err[k]))
    out["topk_w"] = tuple(t.view(T, spec.top_k) for t in out["topk_w"])
    if routing is None:
        del out["topk_w"]
    return out


def check(got, want, what=""):
    """Every element within its bound (plus the smallest normal of the type, for underflow)."""
    val, bound = want
    assert got.shape == val.shape, f"{what}: shape {tuple(got.shape)}, wanted {tuple(val.shape)}"
    tiny = 2.0 ** -126
    off = (got.to(D) - val).abs()
    bad = ~(off <= bound + tiny)
    if bad.any():
        i = int(torch.where(bad, off / (bound + tiny), torch.zeros_like(off)).nan_to_num(nan=1e30).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bound, worst at {i}: got "
                             f"{got.reshape(-1)[i].item():.6g}, wanted {val.reshape(-1)[i].item():.6g} "
                             f"+- {bound.reshape(-1)[i].item():.3g}")


def make_routing(T, spec, gen, dev, experts=None):
    """A random routing over the first `experts` experts (the rest stay empty)."""
    E, k = spec.num_experts, spec.top_k
    idx = torch.stack([torch.randperm(max(experts or E, k), generator=gen)[:k] for _ in range(T)]) if T else \
        torch.zeros(0, k, dtype=torch.long)
    wts = torch.softmax(torch.randn(T, k, generator=gen), -1)
    return routing_of(idx, wts, E, dev)


def routing_of(idx, wts, E, dev):
    flat = idx.reshape(-1)
    order = torch.sort(flat, stable=True).indices.to(torch.int32)
    off = torch.cat([torch.zeros(1, dtype=torch.long), torch.bincount(flat, minlength=E).cumsum(0)]).to(torch.int32)
    return off.to(dev), order.to(dev), wts.to(torch.float32).contiguous().to(dev)
