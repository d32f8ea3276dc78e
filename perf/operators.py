"""Training and serving operators around the expert block: what is measured.

Three operators, each forward and backward:

  linear   y = act(x W^T + b) + r                     latent projections, output projections
  ffn      y = (act(x Wg^T + bg, x Wu^T + bu)) Wd^T + bd (+ r), dense, or a stack of experts
           over routed slots with the routing weights of each token's slots
  norm     layer norm and RMS norm over the last axis

`run` computes them in plain 32-bit torch operations, or, where `own` is set, with
sparse_moe_ffn_gemv_b200.train. Weights are [out, in]; a token's slots are t*k .. t*k + k-1,
grouped by expert with a stable sort (expert_offsets, sorted_slot), as moe_permute writes them.
"""
import functools
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------ cases
def _linear(name, T, n_in, n_out, act="none", bias=False, residual=False, dtype="bf16", backward=False, pad=0):
    return dict(name=name, op="linear", T=T, n_in=n_in, n_out=n_out, act=act, bias=bias, residual=residual,
                dtype=dtype, backward=backward, pad=pad)


def _ffn(name, T, width, inter, E=1, k=1, act="swiglu", interleaved=False, bias=False, residual=False,
         dtype="bf16", backward=False, keep=True, skew=0.0):
    return dict(name=name, op="ffn", T=T, width=width, inter=inter, E=E, k=k, act=act, interleaved=interleaved,
                bias=bias, residual=residual, dtype=dtype, backward=backward, keep=keep, skew=skew)


def _norm(name, T, width, kind="rms", bias=False, dtype="bf16", backward=False, pad=0):
    return dict(name=name, op="norm", T=T, width=width, kind=kind, bias=bias, dtype=dtype, backward=backward,
                pad=pad)


def listed():
    return [
        # serving one token: the latent block's up projection with the shared expert's sum added
        _linear("linear one token", 1, 3584, 7168, residual=True),
        # a prompt through the latent block's down projection
        _linear("linear prompt", 8192, 7168, 3584),
        # a training step's projection with bias and activation, odd token count
        _linear("linear backward odd", 4097, 2880, 2048, act="gelu", bias=True, backward=True),
        # a small 32-bit projection with everything in its epilogue, from a padded buffer
        _linear("linear f32", 77, 192, 320, act="silu", bias=True, residual=True, dtype="f32", pad=16),
        # serving one token through a shared expert
        _ffn("ffn one token", 1, 2048, 768, residual=True, keep=False),
        # a training step's routed experts, many small ones, forward
        _ffn("ffn experts forward", 4096, 2048, 768, E=256, k=8),
        # and their gradients
        _ffn("ffn experts backward", 4096, 2048, 768, E=256, k=8, backward=True),
        # the clamped family: interleaved planes and linear biases, uneven routing
        _ffn("ffn clamped backward", 4001, 2880, 2880, E=32, k=4, act="clamped", interleaved=True, bias=True,
             backward=True, skew=0.5),
        # a wide shared expert's gradients over a large batch
        _ffn("ffn dense backward", 8192, 7168, 2048, backward=True),
        # the tiny 32-bit block
        _ffn("ffn f32 backward", 16, 64, 32, E=8, k=2, dtype="f32", backward=True),
        # the latent norm over a prompt
        _norm("norm rms forward", 8192, 3584),
        # layer norm's gradients over a training batch of the widest hidden size
        _norm("norm layer backward", 8192, 7168, kind="layer", bias=True, backward=True),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["linear", "linear", "ffn", "ffn", "ffn", "norm"])
    back = rng.random() < 0.5
    f32 = rng.random() < 0.2
    dtype = "f32" if f32 else "bf16"
    while True:
        if op == "linear":
            c = _linear("", _log(rng, 1, 600 if f32 else 8192), _log(rng, 64, 512 if f32 else 7168, 8),
                        _log(rng, 64, 512 if f32 else 7168, 8), act=rng.choice(["none", "silu", "gelu"]),
                        bias=rng.random() < 0.5, residual=rng.random() < 0.5, dtype=dtype, backward=back,
                        pad=rng.choice([0, 8, 64]))
        elif op == "norm":
            c = _norm("", _log(rng, 1, 16384), _log(rng, 64, 7168, 8), kind=rng.choice(["layer", "rms"]),
                      bias=rng.random() < 0.5, dtype=dtype, backward=back, pad=rng.choice([0, 8, 64]))
            c["bias"] = c["bias"] and c["kind"] == "layer"
        else:
            E = rng.choice([1, 1, _log(rng, 2, 256)])
            k = 1 if E == 1 else rng.randint(1, min(8, E))
            il = rng.random() < 0.3
            c = _ffn("", _log(rng, 1, 200 if f32 else 8192), _log(rng, 64, 256 if f32 else 7168, 8),
                     _log(rng, 32, 256 if f32 else 2880, 8), E=E, k=k, act=rng.choice(["swiglu", "clamped"]),
                     interleaved=il, bias=rng.random() < 0.4, residual=E == 1 and rng.random() < 0.5, dtype=dtype,
                     backward=back, keep=back or rng.random() < 0.7, skew=rng.choice([0.0, 0.0, 1.0, 2.0]))
        w = work(c)
        # rows that one expert would hold, times the experts: what the plain form's padded products compute
        fair = op != "ffn" or c["E"] == 1 or c["T"] * c["k"] >= c["E"] or c["E"] * c["width"] * c["inter"] < 1 << 28
        if w["flops"] <= 1.4e12 and w["bytes"] <= 4.5e9 and fair:
            del c["name"]
            return c


# ------------------------------------------------------------------------------ inputs
def _dt(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _gen(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1_000_003 * int(seed) + 17)
    return g


def _randn(g, shape, std, dt, mean=0.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std + mean).to(dt)


def _rows(g, T, width, pad, dt, std=1.0):
    """T rows in a buffer whose rows are `pad` values longer."""
    return _randn(g, (T, width + pad), std, dt)[:, :width]


def _planes(g, E, rows, cols, dt):
    w = torch.empty((E, rows, cols), device=DEV, dtype=dt)
    for e in range(E):
        w[e].copy_(torch.randn((rows, cols), generator=g, device=DEV) * 0.02)
    return w


def prepare(case, seed):
    g, dt = _gen(case, seed), _dt(case)
    s = dict(case=case)
    T = case["T"]
    if case["op"] == "linear":
        s["x"] = _rows(g, T, case["n_in"], case["pad"], dt)
        s["w"] = _randn(g, (case["n_out"], case["n_in"]), case["n_in"] ** -0.5, dt)
        s["b"] = _randn(g, (case["n_out"],), 0.2, dt) if case["bias"] else None
        if case["backward"]:
            s["dy"] = _rows(g, T, case["n_out"], case["pad"], dt)
            s["pre"] = _randn(g, (T, case["n_out"]), 1.0, dt) if case["act"] != "none" else None
        else:
            s["r"] = _rows(g, T, case["n_out"], case["pad"], dt) if case["residual"] else None
        return s
    if case["op"] == "norm":
        s["x"] = _rows(g, T, case["width"], case["pad"], dt, 2.0)
        s["w"] = _randn(g, (case["width"],), 0.1, dt, 1.0)
        s["b"] = _randn(g, (case["width"],), 0.1, dt) if case["bias"] else None
        s["eps"] = 1e-6
        if case["backward"]:
            s["dy"] = _rows(g, T, case["width"], case["pad"], dt)
            xf = s["x"].double()
            mu = xf.mean(-1) if case["kind"] == "layer" else torch.zeros(T, device=DEV, dtype=torch.float64)
            var = (xf - mu[:, None]).square().mean(-1)
            s["stats"] = torch.stack([mu, (var + s["eps"]).rsqrt()], -1).float()
        return s
    E, k, K, I = case["E"], case["k"], case["width"], case["inter"]
    s["x"] = _randn(g, (T, K), 1.0, dt)
    w = {}
    if case["interleaved"]:
        w["gate_up_w"] = _planes(g, E, 2 * I, K, dt)
    else:
        w["gate_w"], w["up_w"] = _planes(g, E, I, K, dt), _planes(g, E, I, K, dt)
    w["down_w"] = _planes(g, E, K, I, dt)
    if case["bias"]:
        if case["interleaved"]:
            w["gate_up_b"] = _randn(g, (E, 2 * I), 0.1, dt)
        else:
            w["gate_b"], w["up_b"] = _randn(g, (E, I), 0.1, dt), _randn(g, (E, I), 0.1, dt)
        w["down_b"] = _randn(g, (E, K), 0.1, dt)
    s["w"] = w
    if E > 1:
        # the routing of a trained router: some experts preferred (skew), softmax over the chosen logits
        logits = torch.randn((T, E), generator=g, device=DEV)
        logits += case["skew"] * torch.randn((E,), generator=g, device=DEV)
        top, idx = logits.topk(k, dim=-1)
        s["topk_w"] = torch.softmax(top, -1).contiguous()
        flat = idx.reshape(-1)
        s["sorted_slot"] = torch.sort(flat, stable=True).indices.to(torch.int32)
        counts = torch.bincount(flat, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["cap"] = int(counts.max())
    else:
        s["topk_w"] = s["sorted_slot"] = s["offsets"] = None
        s["cap"] = T
    s["r"] = _randn(g, (T, K), 1.0, dt) if case["residual"] and not case["backward"] else None
    if case["backward"]:
        s["dy"] = _randn(g, (T, K), 1.0, dt)
        # pre-activations of a forward pass, kept for the backward pass: [T*k, 2I] in sorted order
        s["pre"] = _randn(g, (T * k, 2 * I), min(2.0, 0.02 * K ** 0.5), dt)
    return s


# ------------------------------------------------------------------------------ plain forms
LIMIT, ALPHA = 7.0, 1.702


def _act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    return z


def _act_grad(z, act):
    if act == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    return torch.ones_like(z)


def _gated(g, u, act):
    if act == "swiglu":
        return g * torch.sigmoid(g) * u
    gc, uc = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
    return gc * torch.sigmoid(ALPHA * gc) * (uc + 1)


def _gated_grad(g, u, act):
    """(h, dh/dg, dh/du)"""
    if act == "swiglu":
        p = torch.sigmoid(g)
        return g * p * u, p * (1 + g * (1 - p)) * u, g * p
    gc, uc = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
    p = torch.sigmoid(ALPHA * gc)
    dg = p * (1 + ALPHA * gc * (1 - p)) * (uc + 1) * (g <= LIMIT)
    du = gc * p * ((u >= -LIMIT) & (u <= LIMIT))
    return gc * p * (uc + 1), dg, du


def _plain_linear(s):
    c, dt = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    if c["backward"]:
        dz = s["dy"].float()
        if c["act"] != "none":
            dz = dz * _act_grad(s["pre"].float(), c["act"])
        out = [(dz @ w).to(dt), (dz.t() @ x).to(dt)]
        return out + [dz.sum(0).to(dt)] if c["bias"] else out
    z = x @ w.t()
    if c["bias"]:
        z = z + s["b"].float()
    y = _act(z, c["act"])
    if c["residual"]:
        y = y + s["r"].float()
    return [y.to(dt)]


def _plain_norm(s):
    c, dt = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    if not c["backward"]:
        if c["kind"] == "layer":
            mu = x.mean(-1, keepdim=True)
        else:
            mu = torch.zeros_like(x[:, :1])
        d = x - mu
        rstd = 1 / torch.sqrt(d.square().mean(-1, keepdim=True) + s["eps"])
        y = d * rstd * w
        if c["bias"]:
            y = y + s["b"].float()
        return [y.to(dt), torch.cat([mu, rstd], -1)]
    mu, rstd = s["stats"][:, :1], s["stats"][:, 1:]
    xh = (x - mu) * rstd
    dy = s["dy"].float()
    dxh = dy * w
    dx = dxh - xh * (dxh * xh).mean(-1, keepdim=True)
    if c["kind"] == "layer":
        dx = dx - dxh.mean(-1, keepdim=True)
    out = [(dx * rstd).to(dt), (dy * xh).sum(0).to(dt)]
    return out + [dy.sum(0).to(dt)] if c["bias"] else out


def _split(t, interleaved):
    """Gate and up halves of [..., 2I] columns."""
    if interleaved:
        return t[..., 0::2], t[..., 1::2]
    return t.chunk(2, -1)


def _join(g, u, interleaved):
    return torch.stack([g, u], -1).flatten(-2) if interleaved else torch.cat([g, u], -1)


def _gate_up(w, interleaved, suffix):
    """[E, 2I, K] (or the biases [E, 2I]) in 32 bits, in the order of the columns of `pre`."""
    if interleaved:
        return w["gate_up" + suffix].float()
    return torch.cat([w["gate" + suffix].float(), w["up" + suffix].float()], 1)


def _plain_ffn(s):
    """Every expert's rows in one padded batch [E, cap, .]: row p of the sorted order is row
    p - offsets[e] of expert e; rows past an expert's count are zero and go to a spare row."""
    c, w, dt = s["case"], s["w"], s["x"].dtype
    E, k, T, K, il = c["E"], c["k"], c["T"], c["width"], c["interleaved"]
    S = T * k
    at = torch.arange(s["cap"], device=DEV)
    if E > 1:
        off = s["offsets"].long()
        pos = off[:-1, None] + at[None]
        valid = pos < off[1:, None]
        slot = torch.where(valid, s["sorted_slot"].long()[pos.clamp(max=S - 1)], S)
        pos = torch.where(valid, pos, S)
        wt = torch.cat([s["topk_w"].reshape(-1), s["topk_w"].new_zeros(1)])[slot][..., None]
    else:
        pos = slot = at[None]
        valid = pos < S
        wt = torch.ones((1, s["cap"], 1), device=DEV)
    token = slot.clamp(max=S - 1) // k
    x = s["x"].float()[token] * valid[..., None]
    wgu, wd = _gate_up(w, il, "_w"), w["down_w"].float()
    if not c["backward"]:
        gu = x @ wgu.transpose(1, 2)
        if c["bias"]:
            gu = gu + _gate_up(w, il, "_b")[:, None]
        o = _gated(*_split(gu, il), c["act"]) @ wd.transpose(1, 2)
        if c["bias"]:
            o = o + w["down_b"].float()[:, None]
        rows = torch.zeros((S + 1, K), device=DEV)
        rows[slot] = o * wt
        y = rows[:S].view(T, k, K).sum(1)
        if s["r"] is not None:
            y = y + s["r"].float()
        if not c["keep"]:
            return [y.to(dt)]
        pre = torch.zeros((S + 1, gu.shape[-1]), device=DEV)
        pre[pos] = gu
        return [y.to(dt), pre[:S].to(dt)]
    pre = torch.cat([s["pre"].float(), torch.zeros((1, s["pre"].shape[1]), device=DEV)])[pos]
    h, hg, hu = _gated_grad(*_split(pre, il), c["act"])
    h, hg, hu = h * valid[..., None], hg * valid[..., None], hu * valid[..., None]
    dy = s["dy"].float()[token] * valid[..., None]
    dh = dy @ wd
    out = {}
    if E > 1:
        dw = (dh * h).sum(-1)
        if c["bias"]:
            dw = dw + (dy @ w["down_b"].float()[..., None])[..., 0]
        spread = torch.zeros(S + 1, device=DEV)
        spread[slot] = dw
        out["topk_w"] = spread[:S].view(T, k)
    dh = dh * wt
    dgu = _join(dh * hg, dh * hu, il)
    du = torch.zeros((S + 1, K), device=DEV)
    du[slot] = dgu @ wgu
    out["x"] = du[:S].view(T, k, K).sum(1).to(dt)
    out["down_w"] = ((dy * wt).transpose(1, 2) @ h).to(dt)
    dwgu = dgu.transpose(1, 2) @ x
    names = ["gate_up"] if il else ["gate", "up"]
    for n, part in zip(names, dwgu.chunk(len(names), 1)):
        out[n + "_w"] = part.to(dt)
    if c["bias"]:
        out["down_b"] = (dy * wt).sum(1).to(dt)
        for n, part in zip(names, dgu.sum(1).chunk(len(names), 1)):
            out[n + "_b"] = part.to(dt)
    return out


# ------------------------------------------------------------------------------ the framework's calls
@functools.lru_cache(maxsize=None)
def _own_linear(n_in, n_out, act, dtype):
    from sparse_moe_ffn_gemv_b200 import train
    return train.Linear(n_in, n_out, activation=act, dtype=dtype)


@functools.lru_cache(maxsize=None)
def _own_norm(width, kind, eps, dtype):
    from sparse_moe_ffn_gemv_b200 import train
    return train.Norm(width, kind=kind, eps=eps, dtype=dtype)


@functools.lru_cache(maxsize=None)
def _own_ffn(width, inter, E, k, act, il, bias, dtype):
    from sparse_moe_ffn_gemv_b200 import inputs, train
    spec = inputs.MoeSpec(name="", config_id=0, hidden=width, num_experts=E, top_k=k, intermediate=inter,
                          activation="swiglu" if act == "swiglu" else "swiglu_clamped", swiglu_limit=LIMIT,
                          swiglu_alpha=ALPHA, gate_up_interleaved=il, has_expert_bias=bias, act_dtype=dtype,
                          weight_format=dtype)
    return train.GatedFfn(spec)


def _own_run(s):
    c = s["case"]
    if c["op"] == "linear":
        op = _own_linear(c["n_in"], c["n_out"], c["act"], c["dtype"])
        if c["backward"]:
            dx, dw, db = op.backward(s["dy"], s["x"], s["w"], pre=s["pre"], bias_grad=c["bias"])
            return [dx, dw, db] if c["bias"] else [dx, dw]
        return [op.forward(s["x"], s["w"], bias=s["b"], residual=s["r"])]
    if c["op"] == "norm":
        op = _own_norm(c["width"], c["kind"], s["eps"], c["dtype"])
        if c["backward"]:
            dx, dw, db = op.backward(s["dy"], s["x"], s["w"], s["stats"], bias_grad=c["bias"])
            return [dx, dw, db] if c["bias"] else [dx, dw]
        return list(op.forward(s["x"], s["w"], bias=s["b"]))
    op = _own_ffn(c["width"], c["inter"], c["E"], c["k"], c["act"], c["interleaved"], c["bias"], c["dtype"])
    routing = None if c["E"] == 1 else (s["offsets"], s["sorted_slot"], s["topk_w"])
    if c["backward"]:
        return op.backward(s["dy"], s["x"], s["w"], s["pre"], routing=routing)
    y, pre = op.forward(s["x"], s["w"], routing=routing, residual=s["r"], keep=c["keep"])
    return [y, pre] if c["keep"] else [y]


def run(state):
    if own:
        return _own_run(state)
    return {"linear": _plain_linear, "norm": _plain_norm, "ffn": _plain_ffn}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    T = case["T"]
    if case["op"] == "linear":
        N, K = case["n_out"], case["n_in"]
        n = N * K + T * K + T * N + (N if case["bias"] else 0)
        if case["backward"]:
            n += N * K + T * K + (T * N if case["act"] != "none" else 0)
            return dict(bytes=n * es, flops=4 * T * N * K)
        return dict(bytes=(n + (T * N if case["residual"] else 0)) * es, flops=2 * T * N * K)
    if case["op"] == "norm":
        H = case["width"]
        n = 3 * T * H if case["backward"] else 2 * T * H
        n += H * (1 + int(case["bias"])) * (2 if case["backward"] else 1)
        return dict(bytes=n * es + T * 8, flops=(16 if case["backward"] else 8) * T * H)
    E, k, K, I = case["E"], case["k"], case["width"], case["inter"]
    S = T * k
    active = min(E, S)
    weights = 3 * K * I + ((2 * I + K) if case["bias"] else 0)
    pre = 2 * S * I if case["backward"] or case["keep"] else 0
    route = (8 * S + 4 * E) if E > 1 else 0
    if case["backward"]:
        n = active * weights + E * weights + 3 * T * K + pre
        return dict(bytes=n * es + route + (4 * S if E > 1 else 0), flops=12 * S * K * I)
    n = active * weights + 2 * T * K + pre + (T * K if case["residual"] else 0)
    return dict(bytes=n * es + route, flops=6 * S * K * I)


# ------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    D = lambda v: v.to(torch.float64)  # noqa: E731
    if case["op"] == "linear":
        x, w = D(s["x"]), D(s["w"])
        if case["backward"]:
            z = D(s["pre"]) if case["act"] != "none" else None
            dz = D(s["dy"])
            if case["act"] == "silu":
                sg = 1 / (1 + torch.exp(-z))
                dz = dz * (sg + z * sg * (1 - sg))
            elif case["act"] == "gelu":
                dz = dz * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
            res = [torch.einsum("tn,nk->tk", dz, w), torch.einsum("tn,tk->nk", dz, x)]
            return res + [torch.einsum("tn->n", dz)] if case["bias"] else res
        z = torch.einsum("tk,nk->tn", x, w)
        if case["bias"]:
            z += D(s["b"])
        if case["act"] == "silu":
            z = z / (1 + torch.exp(-z))
        elif case["act"] == "gelu":
            z = z * torch.special.ndtr(z)
        return [z + D(s["r"])] if case["residual"] else [z]
    if case["op"] == "norm":
        x, w, n = D(s["x"]), D(s["w"]), case["width"]
        layer = case["kind"] == "layer"
        if not case["backward"]:
            mu = x.sum(-1) / n if layer else x.new_zeros(case["T"])
            var = torch.einsum("th,th->t", x - mu[:, None], x - mu[:, None]) / n
            r = (var + s["eps"]) ** -0.5
            y = torch.einsum("th,t,h->th", x - mu[:, None], r, w)
            if case["bias"]:
                y += D(s["b"])
            return [y, torch.stack([mu, r], 1)]
        mu, r = D(s["stats"])[:, 0], D(s["stats"])[:, 1]
        n_hat = (x - mu[:, None]) * r[:, None]
        dy = D(s["dy"])
        gw = dy * w
        a = gw.sum(-1) / n if layer else x.new_zeros(case["T"])
        b = (gw * n_hat).sum(-1) / n
        dx = r[:, None] * (gw - a[:, None] - n_hat * b[:, None])
        res = [dx, torch.einsum("th,th->h", dy, n_hat)]
        return res + [torch.einsum("th->h", dy)] if case["bias"] else res
    # one expert at a time
    E, k, T, K, I = case["E"], case["k"], case["T"], case["width"], case["inter"]
    w, il = s["w"], case["interleaved"]
    back = case["backward"]
    if E > 1:
        off, order, wt = s["offsets"].tolist(), s["sorted_slot"].long(), D(s["topk_w"]).reshape(-1)
    else:
        off, order, wt = [0, T], torch.arange(T, device=DEV), torch.ones(T, device=DEV, dtype=torch.float64)
    x = D(s["x"])
    grads = {n: torch.zeros(t.shape, device=DEV, dtype=torch.float64) for n, t in w.items()} if back else None
    y = torch.zeros((T, K), device=DEV, dtype=torch.float64)
    pre = torch.zeros((T * k, 2 * I), device=DEV, dtype=torch.float64)
    d_wt = torch.zeros(T * k, device=DEV, dtype=torch.float64)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        slots = order[lo:hi]
        tok = slots // k
        if il:
            wg, wu = D(w["gate_up_w"][e, 0::2]), D(w["gate_up_w"][e, 1::2])
            bg, bu = (D(w["gate_up_b"][e, 0::2]), D(w["gate_up_b"][e, 1::2])) if case["bias"] else (0, 0)
        else:
            wg, wu = D(w["gate_w"][e]), D(w["up_w"][e])
            bg, bu = (D(w["gate_b"][e]), D(w["up_b"][e])) if case["bias"] else (0, 0)
        wd = D(w["down_w"][e])
        if back:
            p = D(s["pre"][lo:hi])
            g, u = (p[:, 0::2], p[:, 1::2]) if il else (p[:, :I], p[:, I:])
        else:
            g, u = x[tok] @ wg.T + bg, x[tok] @ wu.T + bu
            if il:
                pre[lo:hi, 0::2], pre[lo:hi, 1::2] = g, u
            else:
                pre[lo:hi, :I], pre[lo:hi, I:] = g, u
        if case["act"] == "swiglu":
            sg = 1 / (1 + torch.exp(-g))
            gate, dgate, lin, dlin = g * sg, sg + g * sg * (1 - sg), u, 1.0
        else:
            gc = torch.minimum(g, torch.full_like(g, LIMIT))
            sg = 1 / (1 + torch.exp(-ALPHA * gc))
            gate, dgate = gc * sg, (sg + ALPHA * gc * sg * (1 - sg)) * (g <= LIMIT).double()
            lin, dlin = u.clamp(-LIMIT, LIMIT) + 1, (u.abs() <= LIMIT).double()
        h = gate * lin
        sw = wt[slots][:, None]
        if not back:
            o = h @ wd.T
            if case["bias"]:
                o = o + D(w["down_b"][e])
            y.index_add_(0, tok, sw * o)
            continue
        d = D(s["dy"])[tok]
        dh = d @ wd
        d_wt[slots] = (dh * h).sum(1) + ((d @ D(w["down_b"][e])) if case["bias"] else 0)
        dh = dh * sw
        dg, du = dh * dgate * lin, dh * gate * dlin
        y.index_add_(0, tok, dg @ wg + du @ wu)
        grads["down_w"][e] = (d * sw).T @ h
        xs = x[tok]
        parts = [(dg, slice(0, None, 2), "gate"), (du, slice(1, None, 2), "up")]
        for dv, rows, n in parts:
            plane, at = ("gate_up", rows) if il else (n, slice(None))
            grads[plane + "_w"][e, at] = dv.T @ xs
            if case["bias"]:
                grads[plane + "_b"][e, at] = dv.sum(0)
        if case["bias"]:
            grads["down_b"][e] = (d * sw).sum(0)
    if back:
        return dict(grads, x=y, **({"topk_w": d_wt.view(T, k)} if E > 1 else {}))
    if s["r"] is not None:
        y = y + D(s["r"])
    return [y, pre] if case["keep"] else [y]
