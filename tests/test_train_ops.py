"""The training operators on the GPU against their 64-bit definitions (tests/train_ref.py)."""
import pytest
import torch

import train_ref as R
from sparse_moe_ffn_gemv_b200 import inputs
from sparse_moe_ffn_gemv_b200 import moe as M
from sparse_moe_ffn_gemv_b200 import train

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rand(g, shape, dtype, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g) * std + mean).to(DT[dtype]).cuda()


def padded(g, T, n, pad, dtype, std=1.0):
    return rand(g, (T, n + pad), dtype, std)[:, :n]


def ok(op):
    torch.cuda.synchronize()
    assert op.device_status() == 0


# ------------------------------------------------------------------ linear
LINEAR = [  # dtype, T, K, N, act, bias, residual, pad
    ("bf16", 1, 8, 8, "none", False, False, 0),
    ("bf16", 1, 2880, 2048, "gelu", True, True, 8),
    ("bf16", 2, 72, 136, "silu", True, False, 16),
    ("bf16", 3, 1032, 328, "gelu", True, True, 8),
    ("bf16", 4, 2056, 776, "none", False, False, 0),
    ("bf16", 4, 2304, 2304, "silu", True, True, 8),
    ("bf16", 7, 1000, 8, "none", True, True, 0),
    ("bf16", 8, 520, 776, "silu", False, True, 8),
    ("bf16", 17, 200, 264, "gelu", True, True, 8),
    ("bf16", 33, 3584, 96, "none", False, False, 0),
    ("bf16", 64, 64, 1032, "none", True, False, 0),
    ("bf16", 127, 712, 384, "silu", True, True, 40),
    ("bf16", 129, 64, 520, "gelu", False, True, 0),
    ("bf16", 300, 1000, 384, "none", False, True, 8),
    ("bf16", 1030, 328, 776, "silu", True, True, 24),
    ("bf16", 2049, 2048, 264, "gelu", True, False, 0),
    ("bf16", 4096, 512, 2304, "none", True, True, 0),
    ("bf16", 4700, 6152, 1032, "silu", True, True, 8),   # long reductions on 512-row tiles: forward,
    ("bf16", 4700, 1032, 6152, "none", False, False, 0),  # input gradient
    ("bf16", 6200, 1800, 2600, "gelu", True, False, 8),   # and weight gradient
    ("f32", 1, 4, 4, "none", False, False, 0),
    ("f32", 1, 1028, 132, "gelu", True, True, 4),
    ("f32", 33, 100, 60, "silu", True, True, 4),
    ("f32", 130, 68, 132, "gelu", False, False, 12),
    ("f32", 515, 260, 68, "none", True, False, 0),
]


@pytest.mark.parametrize("dtype,T,K,N,act,bias,residual,pad", LINEAR)
def test_linear_forward(dtype, T, K, N, act, bias, residual, pad):
    g = gen(T * 1000 + K + N)
    x, w = padded(g, T, K, pad, dtype), rand(g, (N, K), dtype, K ** -0.5)
    b = rand(g, (N,), dtype, 0.3) if bias else None
    r = padded(g, T, N, pad, dtype) if residual else None
    op = train.Linear(K, N, activation=act, dtype=dtype)
    wide = torch.full((T, N + pad), 7.0, dtype=DT[dtype], device="cuda")
    y, pre = op.forward(x, w, bias=b, residual=r, keep=True, out=wide[:, :N])
    ok(op)
    want_y, want_z = R.linear_forward(x, w, b, r, act)
    R.check(y, want_y, "y")
    R.check(pre, want_z, "pre")
    assert (wide[:, N:] == 7.0).all()  # behind the rows
    R.check(op.forward(x, w, bias=b, residual=r), want_y, "y without pre")


@pytest.mark.parametrize("dtype,T,K,N,act,bias,residual,pad", LINEAR)
def test_linear_backward(dtype, T, K, N, act, bias, residual, pad):
    g = gen(T * 1001 + K + N)
    x, w = padded(g, T, K, pad, dtype), rand(g, (N, K), dtype, K ** -0.5)
    dy = padded(g, T, N, pad, dtype)
    pre = rand(g, (T, N), dtype, 1.5) if act != "none" else None
    op = train.Linear(K, N, activation=act, dtype=dtype)
    dx, dw, db = op.backward(dy, x, w, pre=pre, bias_grad=bias)
    ok(op)
    want = R.linear_backward(dy, x, w, pre, act)
    R.check(dx, want[0], "dx")
    R.check(dw, want[1], "dw")
    if bias:
        R.check(db, want[2], "db")
    # each gradient alone is the same gradient
    only = op.backward(dy, x, w, pre=pre, bias_grad=False, input_grad=False)
    assert only[0] is None and only[2] is None and torch.equal(only[1], dw)
    only = op.backward(dy, x, w, pre=pre, bias_grad=False, weight_grad=False)
    assert only[1] is None and torch.equal(only[0], dx)


def test_linear_residual_may_be_the_output():
    g = gen(5)
    op = train.Linear(256, 320)
    x, w, r = rand(g, (150, 256), "bf16"), rand(g, (320, 256), "bf16", 0.06), rand(g, (150, 320), "bf16")
    want = op.forward(x, w, residual=r)
    buf = r.clone()
    op.forward(x, w, residual=buf, out=buf)
    assert torch.equal(buf, want)


# ------------------------------------------------------------------ gated feed-forward
def spec_of(**kw):
    base = dict(name="t", config_id=0, hidden=64, num_experts=1, top_k=1, intermediate=32)
    base.update(kw)
    base.setdefault("weight_format", base.get("act_dtype", "bf16"))
    return inputs.MoeSpec(**base)


def planes(spec, g):
    E, I, K = spec.num_experts, spec.intermediate, spec.expert_in
    dt = spec.act_dtype
    s = K ** -0.5
    w = {"down_w": rand(g, (E, K, I), dt, I ** -0.5)}
    if spec.gate_up_interleaved:
        w["gate_up_w"] = rand(g, (E, 2 * I, K), dt, s)
    else:
        w["gate_w"], w["up_w"] = rand(g, (E, I, K), dt, s), rand(g, (E, I, K), dt, s)
    if spec.has_expert_bias:
        if spec.gate_up_interleaved:
            w["gate_up_b"] = rand(g, (E, 2 * I), dt, 0.3)
        else:
            w["gate_b"], w["up_b"] = rand(g, (E, I), dt, 0.3), rand(g, (E, I), dt, 0.3)
        w["down_b"] = rand(g, (E, K), dt, 0.3)
    return w


FFN = [  # T, experts with rows (None: all), spec
    (1, None, dict()),
    (1, None, dict(hidden=2048, intermediate=768)),
    (2, None, dict(hidden=1032, intermediate=520, has_expert_bias=True)),
    (3, None, dict(hidden=200, intermediate=72, has_expert_bias=True)),
    (4, None, dict(hidden=264, intermediate=200, gate_up_interleaved=True, has_expert_bias=True,
                   activation="swiglu_clamped", swiglu_limit=0.8)),
    (4, None, dict(hidden=1544, intermediate=1160)),
    (8, None, dict(hidden=520, intermediate=264, gate_up_interleaved=True)),
    (65, None, dict(hidden=72, intermediate=136, activation="swiglu_clamped", swiglu_limit=0.7,
                    gate_up_interleaved=True, has_expert_bias=True)),
    (300, None, dict(hidden=264, intermediate=200, activation="swiglu_clamped", swiglu_limit=1.5)),
    (1025, None, dict(hidden=712, intermediate=328, has_expert_bias=True)),
    (1, None, dict(num_experts=4, top_k=2)),
    (1, None, dict(num_experts=256, top_k=8, hidden=128, intermediate=64)),
    (5, 3, dict(num_experts=8, top_k=3, hidden=72, intermediate=40)),
    (64, 1, dict(num_experts=5, top_k=1, hidden=128, intermediate=64)),
    (129, None, dict(num_experts=3, top_k=2, hidden=136, intermediate=200, has_expert_bias=True)),
    (200, None, dict(num_experts=16, top_k=4, hidden=264, intermediate=136, gate_up_interleaved=True,
                     activation="swiglu_clamped", has_expert_bias=True, swiglu_limit=1.0)),
    (777, 9, dict(num_experts=12, top_k=2, hidden=200, intermediate=328)),
    (900, None, dict(num_experts=4, top_k=3, hidden=320, intermediate=520, activation="swiglu_clamped")),
    (2100, None, dict(num_experts=2, top_k=1, hidden=264, intermediate=264)),
    # large enough for the CTA-pair tiles, the token-wise copies and the bulk stores
    (3001, None, dict(hidden=1096, intermediate=1160, has_expert_bias=True)),
    (2900, None, dict(hidden=1288, intermediate=1032, gate_up_interleaved=True, has_expert_bias=True,
                      activation="swiglu_clamped", swiglu_limit=1.0)),
    (3000, None, dict(num_experts=5, top_k=3, hidden=1096, intermediate=712)),
    (2500, None, dict(num_experts=4, top_k=2, hidden=1160, intermediate=520, gate_up_interleaved=True,
                      has_expert_bias=True, activation="swiglu_clamped", swiglu_limit=1.0)),
    (1500, 50, dict(num_experts=64, top_k=4, hidden=1032, intermediate=264, has_expert_bias=True)),
    (1700, None, dict(num_experts=32, top_k=4, hidden=776, intermediate=328)),
    (650, None, dict(num_experts=3, top_k=2, hidden=4200, intermediate=72, has_expert_bias=True)),
    (700, None, dict(num_experts=2, top_k=2, hidden=8200, intermediate=40)),
    (40, None, dict(num_experts=512, top_k=16, hidden=72, intermediate=40, has_expert_bias=True)),
    (16, None, dict(num_experts=8, top_k=2, act_dtype="f32")),
    (1, None, dict(hidden=100, intermediate=36, act_dtype="f32", has_expert_bias=True)),
    (150, None, dict(hidden=68, intermediate=132, act_dtype="f32", gate_up_interleaved=True, has_expert_bias=True,
                     activation="swiglu_clamped", swiglu_limit=1.0)),
    (140, 5, dict(num_experts=6, top_k=4, hidden=132, intermediate=68, act_dtype="f32", has_expert_bias=True)),
]


def ffn_case(T, experts, kw, seed=0):
    spec = spec_of(**kw)
    g = gen(seed + T * 7 + spec.hidden + 13 * spec.intermediate)
    w = planes(spec, g)
    routing = R.make_routing(T, spec, g, "cuda", experts) if spec.num_experts > 1 else None
    return spec, g, w, routing


@pytest.mark.parametrize("T,experts,kw", FFN)
def test_ffn_forward(T, experts, kw):
    spec, g, w, routing = ffn_case(T, experts, kw)
    x = padded(g, T, spec.hidden, 8, spec.act_dtype)
    r = padded(g, T, spec.hidden, 8, spec.act_dtype) if T % 2 else None
    op = train.GatedFfn(spec)
    y, pre = op.forward(x, w, routing=routing, residual=r)
    ok(op)
    want_y, want_pre = R.ffn_forward(x, w, spec, routing, r)
    R.check(pre, want_pre, "pre")
    R.check(y, want_y, "y")
    y2, none = op.forward(x, w, routing=routing, residual=r, keep=False)
    assert none is None
    R.check(y2, want_y, "y without pre")


@pytest.mark.parametrize("T,experts,kw", FFN)
def test_ffn_backward(T, experts, kw):
    spec, g, w, routing = ffn_case(T, experts, kw, seed=1)
    x, dy = (padded(g, T, spec.hidden, 8, spec.act_dtype) for _ in range(2))
    pre = rand(g, (T * spec.top_k, 2 * spec.intermediate), spec.act_dtype, 1.2)
    op = train.GatedFfn(spec)
    got = op.backward(dy, x, w, pre, routing=routing)
    ok(op)
    want = R.ffn_backward(dy, x, w, pre, spec, routing)
    assert set(got) == set(want)
    for name in want:
        R.check(got[name], want[name], name)
    again = op.backward(dy, x, w, pre, routing=routing)
    assert all(torch.equal(got[n], again[n]) for n in got)  # no sum depends on the run
    less = op.backward(dy, x, w, pre, routing=routing, input_grad=False)
    assert "x" not in less and torch.equal(less["down_w"], got["down_w"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ffn_one_expert_routed_is_the_dense_ffn(dtype):
    """One expert with a routing in token order and weights of one: the dense form's result, up to
    the rounding both may carry; and a permuted routing is the same function."""
    spec = spec_of(hidden=136, intermediate=72, act_dtype=dtype)
    g = gen(6)
    T = 190
    w, x, dy = planes(spec, g), rand(g, (T, 136), dtype), rand(g, (T, 136), dtype)
    op = train.GatedFfn(spec)
    want_y, want_pre = R.ffn_forward(x, w, spec, None, None)
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    order = torch.randperm(T, generator=g).to(torch.int32).cuda()
    routing = (off, order, torch.ones(T, 1, device="cuda"))
    y, pre = op.forward(x, w, routing=routing)
    R.check(y, want_y, "y")
    R.check(pre, tuple(t[order.long()] for t in want_pre), "pre")
    got = op.backward(dy, x, w, pre, routing=routing)
    ok(op)
    want = R.ffn_backward(dy, x, w, pre, spec, routing)
    for name in want:
        R.check(got[name], want[name], name)


def test_ffn_output_rows_may_be_strided():
    spec = spec_of(num_experts=3, top_k=2, hidden=72, intermediate=40)
    g = gen(7)
    for T in (1, 4, 50):
        w, x = planes(spec, g), rand(g, (T, 72), "bf16")
        routing = R.make_routing(T, spec, g, "cuda")
        op = train.GatedFfn(spec)
        wide = torch.full((T, 88), 5.0, dtype=torch.bfloat16, device="cuda")
        y, _ = op.forward(x, w, routing=routing, out=wide[:, 8:80])
        assert y.data_ptr() == wide[:, 8:80].data_ptr()
        R.check(y, R.ffn_forward(x, w, spec, routing, None)[0], "y")
        assert (wide[:, :8] == 5).all() and (wide[:, 80:] == 5).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ffn_same_expert_twice_and_zero_weight(dtype):
    """A token routed twice to one expert, slots of weight zero, every slot on one expert."""
    spec = spec_of(num_experts=4, top_k=2, hidden=72, intermediate=40, act_dtype=dtype, has_expert_bias=True)
    g = gen(3)
    T = 70
    idx = torch.randint(0, 4, (T, 2), generator=g)
    idx[:10, 1] = idx[:10, 0]
    wts = torch.rand(T, 2, generator=g)
    wts[5:20, 1] = 0.0
    for idx in (idx, torch.full((T, 2), 2)):
        routing = R.routing_of(idx, wts, 4, "cuda")
        w, x, dy = planes(spec, g), rand(g, (T, 72), dtype), rand(g, (T, 72), dtype)
        op = train.GatedFfn(spec)
        y, pre = op.forward(x, w, routing=routing)
        R.check(y, R.ffn_forward(x, w, spec, routing, None)[0], "y")
        got = op.backward(dy, x, w, pre, routing=routing)
        ok(op)
        want = R.ffn_backward(dy, x, w, pre, spec, routing)
        for name in want:
            R.check(got[name], want[name], name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ffn_planes_of_experts_without_rows_are_not_used(dtype):
    """NaN and infinities in the planes of experts that hold no row reach nothing."""
    spec = spec_of(num_experts=6, top_k=2, hidden=136, intermediate=72, act_dtype=dtype, has_expert_bias=True)
    g = gen(9)
    T = 90
    w = planes(spec, g)
    routing = R.make_routing(T, spec, g, "cuda", experts=3)
    clean = {n: t.clone() for n, t in w.items()}
    for t in w.values():
        t[3:] = float("nan")
        t[5] = float("inf")
    x, dy = rand(g, (T, 136), dtype), rand(g, (T, 136), dtype)
    op = train.GatedFfn(spec)
    y, pre = op.forward(x, w, routing=routing)
    y0, pre0 = op.forward(x, clean, routing=routing)
    assert torch.equal(y, y0) and torch.equal(pre, pre0)
    a, b = op.backward(dy, x, w, pre, routing=routing), op.backward(dy, x, clean, pre, routing=routing)
    ok(op)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    assert (a["down_w"][3:] == 0).all() and (a["gate_b"][3:] == 0).all()


def test_ffn_infinite_weight_stays_in_its_expert():
    """An infinity in one expert's plane reaches the gradients of that expert's rows only."""
    spec = spec_of(num_experts=3, top_k=1, hidden=64, intermediate=64)
    g = gen(10)
    T = 100
    idx = torch.arange(T)[:, None] % 3
    routing = R.routing_of(idx, torch.ones(T, 1), 3, "cuda")
    w = planes(spec, g)
    x, dy = rand(g, (T, 64), "bf16"), rand(g, (T, 64), "bf16")
    op = train.GatedFfn(spec)
    _, pre = op.forward(x, w, routing=routing)
    ref = op.backward(dy, x, w, pre, routing=routing)
    w["down_w"][1, 5, 7] = float("inf")
    got = op.backward(dy, x, w, pre, routing=routing)
    ok(op)
    for e in (0, 2):
        for n in ("gate_w", "up_w", "down_w"):
            assert torch.equal(got[n][e], ref[n][e])
    # within the expert: column 7 of dh is infinite, and with it row 7 of the gate and up gradients
    assert torch.equal(got["down_w"][1], ref["down_w"][1])
    rows = torch.ones(64, dtype=torch.bool)
    rows[7] = False
    assert torch.equal(got["gate_w"][1][rows.cuda()], ref["gate_w"][1][rows.cuda()])
    assert not torch.isfinite(got["gate_w"][1, 7]).any()


def test_ffn_nan_input_stays_in_its_token():
    spec = spec_of(num_experts=2, top_k=1, hidden=64, intermediate=64, activation="swiglu_clamped")
    g = gen(11)
    T = 40
    routing = R.routing_of((torch.arange(T) % 2)[:, None], torch.ones(T, 1), 2, "cuda")
    w, x = planes(spec, g), rand(g, (T, 64), "bf16")
    op = train.GatedFfn(spec)
    ref, _ = op.forward(x, w, routing=routing)
    x[6, 3] = float("nan")
    y, pre = op.forward(x, w, routing=routing)
    ok(op)
    assert torch.isnan(y[6]).all() and torch.isnan(pre[3]).all()  # token 6 is row 3 of expert 0
    keep = torch.arange(T) != 6
    assert torch.equal(y[keep.cuda()], ref[keep.cuda()])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ffn_dropped_slots(dtype):
    """Slots that moe_permute dropped (expert id out of range): no output, zero gradient, their
    rows of pre left as they were."""
    spec = spec_of(num_experts=4, top_k=2, hidden=64, intermediate=32, act_dtype=dtype)
    cfg = M.config_from_spec(spec)
    g = gen(12)
    T = 30
    idx = torch.randint(0, 4, (T, 2), generator=g).to(torch.int32)
    idx[4, 1] = 99
    idx[7] = -1
    wts = torch.rand(T, 2, generator=g).cuda()
    ws = torch.zeros(M.moe_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    off, ss, sp = torch.zeros(5, **i32), torch.zeros(T * 2, **i32), torch.zeros(T * 2, **i32)
    M.moe_permute(cfg, idx.cuda(), T, off, ss, sp, ws)
    assert M.moe_read_device_status(ws) == M.STATUS_CODE["MOE_ERR_DEVICE_CHECK"]
    n = int(off[-1])
    assert n == T * 2 - 3
    w, x, dy = planes(spec, g), rand(g, (T, 64), dtype), rand(g, (T, 64), dtype)
    op = train.GatedFfn(spec)
    y, pre = op.forward(x, w, routing=(off, ss, wts))
    want_y, want_pre = R.ffn_forward(x, w, spec, (off, ss, wts), None)
    R.check(y, want_y, "y")
    R.check(pre[:n], tuple(t[:n] for t in want_pre), "pre")
    assert (y[7] == 0).all()
    got = op.backward(dy, x, w, pre, routing=(off, ss, wts))
    ok(op)
    want = R.ffn_backward(dy, x, w, pre, spec, (off, ss, wts))
    for name in want:
        R.check(got[name], want[name], name)
    assert got["topk_w"][4, 1] == 0 and (got["topk_w"][7] == 0).all() and (got["x"][7] == 0).all()


def test_ffn_bad_permutations_are_reported():
    """Slot ids and offsets out of range: the rows are dropped and the status says so."""
    spec = spec_of(num_experts=4, top_k=2, hidden=64, intermediate=64)
    g = gen(13)
    T = 20
    off, ss, wts = R.make_routing(T, spec, g, "cuda")
    w, x = planes(spec, g), rand(g, (T, 64), "bf16")
    op = train.GatedFfn(spec)
    want, _ = op.forward(x, w, routing=(off, ss, wts))
    bad = ss.clone()
    slot = int(bad[7])
    bad[7] = 2 ** 30
    y, _ = op.forward(x, w, routing=(off, bad, wts))
    torch.cuda.synchronize()
    assert op.device_status() == M.STATUS_CODE["MOE_ERR_DEVICE_CHECK"]
    keep = (torch.arange(T) != slot // 2).cuda()
    assert torch.equal(y[keep], want[keep])
    for wrong in (off.flip(0).contiguous(), off + 100, off - 1):
        y, _ = op.forward(x, w, routing=(wrong, ss, wts))
        torch.cuda.synchronize()
        assert op.device_status() == M.STATUS_CODE["MOE_ERR_DEVICE_CHECK"]
        assert (y == 0).all()
    assert op.device_status() == 0  # read and cleared


@pytest.mark.parametrize("T,width,kw", [
    (20, 64, {}), (20, 64, dict(has_expert_bias=True)), (2100, 1024, {}), (2100, 1024, dict(has_expert_bias=True)),
    (20, 64, dict(act_dtype="f32")), (2100, 1024, dict(act_dtype="f32", has_expert_bias=True)),
])
def test_ffn_slot_that_stands_twice_is_reported(T, width, kw):
    """One slot in place of another: the status says so, the other tokens keep their results, and
    no value that was in the workspace before gets into a gradient."""
    spec = spec_of(num_experts=4, top_k=2, hidden=width, intermediate=64, **kw)
    g = gen(15)
    off, ss, wts = R.make_routing(T, spec, g, "cuda")
    w, x, dy = planes(spec, g), rand(g, (T, width), spec.act_dtype), rand(g, (T, width), spec.act_dtype)
    op = train.GatedFfn(spec)
    want, _ = op.forward(x, w, routing=(off, ss, wts))
    ok(op)
    bad = ss.clone()
    bad[11] = bad[int(off[2]) + 3]
    gone = torch.tensor([int(bad[11]) // 2, int(ss[11]) // 2])
    keep = torch.ones(T, dtype=torch.bool)
    keep[gone] = False
    for _ in range(2):
        poison = torch.full((1 << 26,), float("nan"), device="cuda")  # what the next workspace holds
        del poison
        y, pre = op.forward(x, w, routing=(off, bad, wts))
        assert op.device_status() == M.STATUS_CODE["MOE_ERR_DEVICE_CHECK"]
        assert torch.equal(y[keep.cuda()], want[keep.cuda()])
        poison = torch.full((1 << 26,), float("nan"), device="cuda")
        del poison
        got = op.backward(dy, x, w, torch.nan_to_num(pre), routing=(off, bad, wts))
        assert op.device_status() == M.STATUS_CODE["MOE_ERR_DEVICE_CHECK"]
        for name, t in got.items():
            assert torch.isfinite(t).all(), name


@pytest.mark.parametrize("T,kw", [
    (1, dict(num_experts=1, top_k=1)), (4, dict(num_experts=1, top_k=1)), (300, dict(num_experts=1, top_k=1)),
    (50, dict(num_experts=4, top_k=2)), (60, dict(num_experts=1, top_k=1, act_dtype="f32")),
    (2100, dict(num_experts=4, top_k=2, hidden=1024)),
])
def test_ffn_output_may_be_its_input_and_residual(T, kw):
    spec = spec_of(**{**dict(hidden=72, intermediate=40), **kw})
    g = gen(16)
    w, x = planes(spec, g), rand(g, (T, spec.expert_in), spec.act_dtype)
    routing = None if spec.num_experts == 1 else R.make_routing(T, spec, g, "cuda")
    op = train.GatedFfn(spec)
    want, _ = op.forward(x, w, routing=routing, residual=x)
    got = x.clone()
    op.forward(got, w, routing=routing, residual=got, out=got)
    ok(op)
    assert torch.equal(got, want)


def test_linear_output_beside_its_input():
    """x and y as column slices of one buffer; y over x is refused."""
    g = gen(17)
    for T, dtype in ((1, "bf16"), (3, "bf16"), (400, "bf16"), (90, "f32")):
        x, w = rand(g, (T, 72), dtype), rand(g, (72, 72), dtype)
        op = train.Linear(72, 72, dtype=dtype)
        both = torch.zeros((T, 160), dtype=DT[dtype], device="cuda")
        both[:, 8:80] = x
        y = op.forward(both[:, 8:80], w, out=both[:, 80:152])
        ok(op)
        assert torch.equal(y, op.forward(x, w)) and torch.equal(both[:, 8:80], x) and (both[:, 152:] == 0).all()
        with pytest.raises(M.MoeError):
            op.forward(both[:, 8:80], w, out=both[:, 8:80])
        with pytest.raises(M.MoeError):
            op.forward(both[:, 8:80], w, out=both[:, 72:144])


# ------------------------------------------------------------------ norm
NORM = [  # dtype, T, H, kind, bias, pad
    ("bf16", 1, 8, "rms", False, 0), ("bf16", 1, 3584, "rms", False, 0), ("bf16", 3, 64, "layer", True, 8),
    ("bf16", 33, 1000, "layer", False, 16), ("bf16", 257, 2880, "rms", False, 8), ("bf16", 1000, 768, "layer", True, 0),
    ("bf16", 70, 7168, "layer", True, 0), ("bf16", 5, 16384, "rms", False, 0), ("bf16", 4, 20008, "layer", True, 8),
    ("bf16", 3000, 136, "rms", False, 0),
    ("f32", 1, 4, "layer", True, 0), ("f32", 40, 1004, "rms", False, 4), ("f32", 130, 2048, "layer", True, 0),
    ("f32", 9, 9000, "layer", False, 4), ("f32", 2, 12004, "rms", False, 0),
]


@pytest.mark.parametrize("dtype,T,H,kind,bias,pad", NORM)
@pytest.mark.parametrize("shift", [0.0, 30.0])
def test_norm_forward(dtype, T, H, kind, bias, pad, shift):
    g = gen(T + H)
    x = (padded(g, T, H, pad, "f32", 2.0) + shift).to(DT[dtype])
    x = torch.cat([x, torch.zeros_like(x[:, :pad])], 1)[:, :H] if pad else x
    w, b = rand(g, (H,), dtype, 0.3, 1.0), rand(g, (H,), dtype, 0.3) if bias else None
    op = train.Norm(H, kind=kind, eps=1e-5, dtype=dtype)
    y, stats = op.forward(x, w, bias=b)
    want_y, want_s = R.norm_forward(x, w, b, 1e-5, kind)
    R.check(stats, want_s, "stats")
    R.check(y, want_y, "y")
    xc = x.clone()
    op.forward(xc, w, bias=b, out=xc)  # in place
    assert torch.equal(xc, y)


def test_norm_of_a_constant_row_is_the_bias():
    op = train.Norm(512, kind="layer", eps=1e-5)
    w, b = torch.ones(512, dtype=torch.bfloat16, device="cuda"), torch.full((512,), 0.5, dtype=torch.bfloat16, device="cuda")
    y, _ = op.forward(torch.full((3, 512), 17.0, dtype=torch.bfloat16, device="cuda"), w, bias=b)
    assert (y == 0.5).all()
    y, stats = op.forward(torch.zeros((3, 512), dtype=torch.bfloat16, device="cuda"), w, bias=b)
    assert (y == 0.5).all() and torch.isfinite(stats).all()


@pytest.mark.parametrize("dtype,T,H,kind,bias,pad", NORM)
def test_norm_backward(dtype, T, H, kind, bias, pad):
    g = gen(2 * T + H)
    x, dy = padded(g, T, H, pad, dtype, 2.0), padded(g, T, H, pad, dtype)
    w = rand(g, (H,), dtype, 0.3, 1.0)
    op = train.Norm(H, kind=kind, eps=1e-5, dtype=dtype)
    _, stats = op.forward(x, w)
    dx, dw, db = op.backward(dy, x, w, stats, bias_grad=bias)
    want = R.norm_backward(dy, x, w, stats, kind)
    R.check(dx, want[0], "dx")
    R.check(dw, want[1], "dw")
    if bias:
        R.check(db, want[2], "db")
    assert (db is None) == (not bias)
    _, dw2, _ = op.backward(dy, x, w, stats, bias_grad=bias, input_grad=False)
    R.check(dw2, want[1], "dw alone")


# ------------------------------------------------------------------ against differences
def directional(loss, t, direction, eps):
    """Central difference of loss along direction at t."""
    return (loss(t + eps * direction) - loss(t - eps * direction)) / (2 * eps)


def test_gradients_against_differences():
    """f32 forward passes differenced along random directions. The difference quotient is off by
    the third derivative times eps^2 / 6 and by the forward's rounding over eps; with unit-scale
    data, eps = 1e-2 and losses of order 10 both stay below 1e-3 of the gradient's scale."""
    g = gen(21)
    T, K, N, I = 12, 20, 24, 16
    dot = lambda a, b: float((a.double() * b.double()).sum())  # noqa: E731
    close = lambda a, b, scale: abs(a - b) <= 2e-3 * scale  # noqa: E731
    unit = lambda shape: torch.nn.functional.normalize(rand(g, shape, "f32").reshape(-1), dim=0).reshape(shape)  # noqa: E731
    # linear
    for act in ("none", "silu", "gelu"):
        op = train.Linear(K, N, activation=act, dtype="f32")
        t = dict(x=rand(g, (T, K), "f32"), w=rand(g, (N, K), "f32", 0.3), b=rand(g, (N,), "f32"))
        c = rand(g, (T, N), "f32")
        _, pre = op.forward(t["x"], t["w"], bias=t["b"], keep=True)
        grads = dict(zip("xwb", op.backward(c, t["x"], t["w"], pre=pre if act != "none" else None)))
        for n in "xwb":
            u = unit(t[n].shape)
            f = lambda v: dot(op.forward(*[v if m == n else t[m] for m in "xw"], bias=v if n == "b" else t["b"]), c)  # noqa: B023,E731
            assert close(directional(f, t[n], u, 1e-2), dot(grads[n], u), float(grads[n].norm())), (act, n)
    # norm
    for kind in ("layer", "rms"):
        op = train.Norm(K, kind=kind, dtype="f32")
        x, w, c = rand(g, (T, K), "f32"), rand(g, (K,), "f32", 0.3, 1.0), rand(g, (T, K), "f32")
        _, stats = op.forward(x, w)
        dx, dw, _ = op.backward(c, x, w, stats)
        for v, grad, f in ((x, dx, lambda v: dot(op.forward(v, w)[0], c)), (w, dw, lambda v: dot(op.forward(x, v)[0], c))):
            u = unit(v.shape)
            assert close(directional(f, v, u, 1e-2), dot(grad, u), float(grad.norm())), kind
    # gated feed-forward, routed
    for act in ("swiglu", "swiglu_clamped"):
        spec = spec_of(num_experts=3, top_k=2, hidden=K, intermediate=I, act_dtype="f32", activation=act,
                       has_expert_bias=True, swiglu_limit=30.0)
        w, x, c = planes(spec, g), rand(g, (T, K), "f32"), rand(g, (T, K), "f32")
        off, ss, wts = R.make_routing(T, spec, g, "cuda")
        op = train.GatedFfn(spec)
        _, pre = op.forward(x, w, routing=(off, ss, wts))
        grads = op.backward(c, x, w, pre, routing=(off, ss, wts))
        for n in grads:
            base = x if n == "x" else wts if n == "topk_w" else w[n]
            u = unit(base.shape)
            def f(v):
                ww = dict(w, **({n: v} if n in w else {}))  # noqa: B023
                y, _ = op.forward(v if n == "x" else x, ww, routing=(off, ss, v if n == "topk_w" else wts))  # noqa: B023
                return dot(y, c)  # noqa: B023
            assert close(directional(f, base, u, 1e-2), dot(grads[n], u), float(grads[n].norm())), (act, n)


# ------------------------------------------------------------------ together
def latent_step(spec, w, x, dy, routing):
    """Forward and backward of a latent block with its shared expert, at a fixed routing."""
    H, L = spec.hidden, spec.latent_dim
    down, up = train.Linear(H, L), train.Linear(L, H)
    ffn = train.GatedFfn(spec)
    shared_spec = spec_of(hidden=H, intermediate=spec.shared_intermediate)
    shared = train.GatedFfn(shared_spec)
    sw = {"gate_w": w["shared_gate_w"], "up_w": w["shared_up_w"], "down_w": w["shared_down_w"]}
    norm = train.Norm(L, kind="rms", eps=spec.rms_eps)
    z = down.forward(x, w["latent_down_w"])
    yr, pre = ffn.forward(z, w, routing=routing)
    n, stats = norm.forward(yr, w["latent_norm_w"])
    s, spre = shared.forward(x, sw)
    y = up.forward(n, w["latent_up_w"], residual=s)
    g = {}
    dn, g["latent_up_w"], _ = up.backward(dy, n, w["latent_up_w"], bias_grad=False)
    gs = shared.backward(dy, x, sw, spre)
    dyr, g["latent_norm_w"], _ = norm.backward(dn, yr, w["latent_norm_w"], stats)
    ge = ffn.backward(dyr, z, w, pre, routing=routing)
    dx, g["latent_down_w"], _ = down.backward(ge["x"], x, w["latent_down_w"], bias_grad=False)
    g.update({"shared_" + k: gs[k] for k in ("gate_w", "up_w", "down_w")})
    g.update({k: ge[k] for k in ("gate_w", "up_w", "down_w", "topk_w")})
    g["x"] = dx.float() + gs["x"].float()
    for op in (down, up, ffn, shared):
        assert op.device_status() == 0
    return y, g


def test_latent_block_training_step():
    """The operators as a latent block's training step, against torch.autograd in 64 bits, and
    its forward against the block's own moe_block_forward. Every intermediate is rounded to
    bf16 (2^-9 rms each, about eight of them on the longest path, amplified by the RMS norm's
    unit gain): relative 2-norm errors stay below sqrt(16) * 2^-8 = 1.6e-2."""
    spec = inputs.MoeSpec(name="latent", config_id=11, hidden=256, num_experts=8, top_k=2, intermediate=128,
                          scoring="sigmoid", norm_topk_prob=True, shared_mode="add", shared_intermediate=192,
                          latent_dim=128, latent_use_norm=True)
    T = 300
    w = {k: v.cuda() for k, v in inputs.make_weights(spec).items()}
    for k in list(w):
        if k.endswith("_w") and k not in ("router_w", "latent_norm_w"):
            w[k] = (w[k].float() * 4).to(w[k].dtype)
    x = inputs.make_x(spec, T).cuda()
    g = gen(31)
    dy = rand(g, (T, 256), "bf16")
    # the block's own router and permutation
    block = M.MoeBlock(spec, w, T)
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, wts = torch.empty(T, 2, **i32), torch.empty(T, 2, dtype=torch.float32, device="cuda")
    off, ss, sp = torch.empty(9, **i32), torch.empty(2 * T, **i32), torch.empty(2 * T, **i32)
    M.moe_route(block.cfg, block.w, x, T, idx, wts, None, block.ws)
    M.moe_permute(block.cfg, idx, T, off, ss, sp, block.ws)
    y, grads = latent_step(spec, w, x, dy, (off, ss, wts))
    rel = lambda a, b: float((a.double() - b.double()).norm() / b.double().norm())  # noqa: E731
    assert rel(y, block.forward(x)) < 1.6e-2
    # 64-bit autograd of the same formulas
    p = {k: v.double().requires_grad_() for k, v in w.items() if k != "router_w"}
    x64, wt64 = x.double().requires_grad_(), wts.double().requires_grad_()
    silu = torch.nn.functional.silu
    z = x64 @ p["latent_down_w"].T
    yr = torch.zeros_like(z)
    for e in range(8):
        t, j = torch.where(idx == e)
        h = silu(z[t] @ p["gate_w"][e].T) * (z[t] @ p["up_w"][e].T)
        yr = yr.index_add(0, t, wt64[t, j][:, None] * (h @ p["down_w"][e].T))
    n = yr * (yr.square().mean(-1, keepdim=True) + spec.rms_eps) ** -0.5 * p["latent_norm_w"]
    s = (silu(x64 @ p["shared_gate_w"].T) * (x64 @ p["shared_up_w"].T)) @ p["shared_down_w"].T
    y64 = n @ p["latent_up_w"].T + s
    y64.backward(dy.double())
    assert rel(y, y64) < 1.6e-2
    for k, v in grads.items():
        ref = x64.grad if k == "x" else wt64.grad if k == "topk_w" else p[k].grad
        assert rel(v, ref) < 1.6e-2, k


# ------------------------------------------------------------------ streams, graphs, sizes
def test_no_tokens():
    lin, norm = train.Linear(64, 128, activation="silu"), train.Norm(64, kind="layer")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, w = torch.empty(0, 64, **bf), torch.ones(128, 64, **bf)
    assert lin.forward(x, w).shape == (0, 128)
    dx, dw, db = lin.backward(torch.empty(0, 128, **bf), x, w, pre=torch.empty(0, 128, **bf))
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    y, stats = norm.forward(x, w[0])
    dx, dw, db = norm.backward(y, x, w[0], stats)
    assert (dw == 0).all() and (db == 0).all()
    spec = spec_of(num_experts=3, top_k=2, has_expert_bias=True)
    p = planes(spec, gen(1))
    routing = R.make_routing(0, spec, gen(1), "cuda")
    ffn = train.GatedFfn(spec)
    y, pre = ffn.forward(x, p, routing=routing)
    got = ffn.backward(y, x, p, pre, routing=routing)
    torch.cuda.synchronize()
    assert all((got[n] == 0).all() for n in p)


def steps():
    """(name, call) of every operator and direction on fixed inputs."""
    g = gen(41)
    spec = spec_of(num_experts=6, top_k=2, hidden=192, intermediate=136, has_expert_bias=True)
    w = planes(spec, g)
    T = 333
    x, dy = rand(g, (T, 192), "bf16"), rand(g, (T, 192), "bf16")
    routing = R.make_routing(T, spec, g, "cuda")
    lw, lb, pre_l = rand(g, (320, 192), "bf16", 0.07), rand(g, (320,), "bf16"), rand(g, (T, 320), "bf16")
    ldy = rand(g, (T, 320), "bf16")
    pre = rand(g, (2 * T, 272), "bf16")
    ffn, lin, norm = train.GatedFfn(spec), train.Linear(192, 320, activation="gelu"), train.Norm(192, kind="layer")
    stats = norm.forward(x, lw[0])[1]
    return [
        ("linear", lambda: [lin.forward(x, lw, bias=lb, residual=ldy)]),
        ("linear one", lambda: [lin.forward(x[:1], lw, bias=lb, residual=ldy[:1])]),
        ("linear back", lambda: list(lin.backward(ldy, x, lw, pre=pre_l))),
        ("ffn", lambda: list(ffn.forward(x, w, routing=routing))),
        ("ffn back", lambda: list(ffn.backward(dy, x, w, pre, routing=routing).values())),
        ("norm", lambda: list(norm.forward(x, lw[0], bias=lw[1]))),
        ("norm back", lambda: list(norm.backward(dy, x, lw[0], stats))),
    ]


def test_refusals_name_the_tensor():
    """Shapes, types and strides that the library would misread are refused before the call."""
    bf = dict(dtype=torch.bfloat16, device="cuda")
    lin = train.Linear(64, 128)
    x, w = torch.zeros(5, 64, **bf), torch.zeros(128, 64, **bf)
    for bad, name in ((dict(x=x.float()), "x"), (dict(x=x[:, :32]), "x"), (dict(x=torch.zeros(64, 5, **bf).t()), "x"),
                      (dict(x=x.cpu()), "x"), (dict(w=w[:64]), "w"), (dict(w=torch.zeros(64, 128, **bf).t()), "w"),
                      (dict(bias=torch.zeros(64, **bf)), "bias"), (dict(residual=torch.zeros(4, 128, **bf)), "residual"),
                      (dict(out=torch.zeros(5, 64, **bf)), "out")):
        with pytest.raises(ValueError, match=name):
            lin.forward(**{**dict(x=x, w=w), **bad})
    with pytest.raises(M.MoeError) as e:  # a row stride that is no multiple of 16 bytes
        lin.forward(torch.zeros(5, 68, **bf)[:, :64], w)
    assert e.value.name == "MOE_ERR_INVALID_ARGUMENT"
    with pytest.raises(M.MoeError) as e:
        lin.forward(torch.zeros(5, 72, **bf)[:, 1:65], w)  # rows that do not begin at 16 bytes
    assert e.value.name == "MOE_ERR_INVALID_ARGUMENT"
    with pytest.raises(M.MoeError) as e:
        train.Linear(64, 128, activation="silu").backward(torch.zeros(5, 128, **bf), x, w)
    assert e.value.name == "MOE_ERR_MISSING_TENSOR"
    ffn = train.GatedFfn(spec_of(num_experts=2, top_k=1))
    p = planes(ffn.spec, gen(1))
    with pytest.raises(ValueError, match="routing"):
        ffn.forward(x, p)
    with pytest.raises(M.MoeError, match="down_w"):
        ffn.forward(x, {k: v for k, v in p.items() if k != "down_w"}, routing=R.make_routing(5, ffn.spec, gen(1), "cuda"))
    with pytest.raises(ValueError, match="bias"):
        train.Norm(64).backward(x, x, w[0], torch.zeros(5, 2, device="cuda"), bias_grad=True)
    for make in (lambda: train.Linear(64, 128, activation="relu"), lambda: train.Linear(64, 128, dtype="fp16"),
                 lambda: train.Norm(64, kind="batch"), lambda: train.Linear(64, 128, device="cpu")):
        with pytest.raises(ValueError):
            make()
    with pytest.raises(M.MoeError):
        train.Linear(60, 128)
    with pytest.raises(M.MoeError):
        train.GatedFfn(spec_of(hidden=128, intermediate=64, weight_format="mxfp4", group_size=32))


def test_calls_on_two_streams_at_once():
    calls = steps()
    want = [[t.clone() for t in c()] for _, c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _, c in calls * 3:
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(c())
    torch.cuda.synchronize()
    for g in got:
        for k, out in enumerate(g):
            for a, b in zip(out, want[k % len(calls)]):
                assert torch.equal(a, b), calls[k % len(calls)][0]


def test_explicit_stream_argument():
    op = train.Linear(192, 320)
    g = gen(43)
    x, w = rand(g, (100, 192), "bf16"), rand(g, (320, 192), "bf16")
    want = op.forward(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = op.forward(x, w, stream=s)
    s.synchronize()
    assert torch.equal(y, want)


def test_captured_and_replayed_in_two_graphs():
    calls = steps()
    want = [[t.clone() for t in c()] for _, c in calls]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = [c() for _, c in calls]
        graphs.append((g, outs))
    for _ in range(2):
        for g, outs in graphs:
            for o in outs:
                for t in o:
                    t.zero_()
            g.replay()
            torch.cuda.synchronize()
            for (name, _), o, w in zip(calls, outs, want):
                assert all(torch.equal(a, b) for a, b in zip(o, w)), name

def chain(g, dtype, T, sync):
    """Operators of every form, one on the other's results, whose inputs are overwritten as soon as
    the call that reads them is launched. `sync` waits after each."""
    H = 264
    spec = spec_of(num_experts=6, top_k=2, hidden=H, intermediate=72, act_dtype=dtype, has_expert_bias=True)
    dense = spec_of(hidden=H, intermediate=136, act_dtype=dtype)
    lin, ffn, mlp, norm = (train.Linear(H, H, "gelu", dtype=dtype), train.GatedFfn(spec), train.GatedFfn(dense),
                           train.Norm(H, "layer", dtype=dtype))
    w, b = rand(g, (H, H), dtype, H ** -0.5), rand(g, (H,), dtype)
    wf, wm = planes(spec, g), planes(dense, g)
    off, slots, wts = R.make_routing(T, spec, g, "cuda")
    start = rand(g, (T, H), dtype)
    x, nan = torch.empty_like(start), float("nan")

    def step(y):
        if sync:
            torch.cuda.synchronize()
        return y

    def run():
        out = []
        x.copy_(start)                                   # a copy before, a fill after the call
        y, stats = step(norm.forward(x, b, bias=b))
        z, pre = step(lin.forward(y, w, bias=b, keep=True))
        u, _ = step(mlp.forward(z, wm, residual=y, keep=False))
        v, vpre = step(ffn.forward(u, wf, routing=(off, slots, wts), residual=u))
        gf = step(ffn.backward(v, u, wf, vpre, routing=(off, slots, wts)))
        v.fill_(nan)
        vpre.fill_(nan)
        dz = gf["x"]
        dy, dw, db = step(lin.backward(dz, y, w, pre))
        dz.fill_(nan)
        dx, dn, dnb = step(norm.backward(dy, x, b, stats))
        x.fill_(nan)
        y.fill_(nan)
        dy.fill_(nan)
        out += [u, dw, db, dx, dn, dnb, gf["topk_w"]] + [gf[n] for n in sorted(wf)]
        return out

    return run


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 3, 40, 700])
def test_calls_one_behind_the_other(dtype, T):
    """Launches overlap their neighbours' ends; the results are those of calls with a wait between."""
    want = chain(gen(31), dtype, T, True)()
    run = chain(gen(31), dtype, T, False)
    for _ in range(20):
        for a, b in zip(run(), want):
            assert torch.isfinite(b).all() and torch.equal(a, b)
    # the same as a graph, whose calls follow copies, fills and a join of two branches
    stream, side = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    flag = torch.zeros(1 << 20, device="cuda")
    with torch.cuda.stream(stream):
        run()
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            side.wait_stream(stream)
            with torch.cuda.stream(side):
                flag.zero_()
            stream.wait_stream(side)
            got = run()
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_ffn_offsets_past_32_bits():
    """Routed rows whose element offsets pass 2^31: 40,000 tokens in 8 slots each of 7168 values.
    A few tokens are not zero; the others' rows and gradients are zeros."""
    spec = spec_of(num_experts=9, top_k=8, hidden=7168, intermediate=64)
    T = 40_000
    g = gen(52)
    w = planes(spec, g)
    idx = (torch.arange(T)[:, None] + torch.arange(8)) % 9
    routing = R.routing_of(idx, torch.rand(T, 8, generator=g), 9, "cuda")
    rows = torch.tensor([0, 17, 20_001, 39_990, 39_999])
    x = torch.zeros((T, 7168), dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros_like(x)
    x[rows.cuda()], dy[rows.cuda()] = rand(g, (5, 7168), "bf16"), rand(g, (5, 7168), "bf16")
    op = train.GatedFfn(spec)
    y, pre = op.forward(x, w, routing=routing)
    got = op.backward(dy, x, w, pre, routing=routing)
    ok(op)
    # the same five tokens alone
    sub = R.routing_of(idx[rows], routing[2].cpu()[rows], 9, "cuda")
    xs, dys = x[rows.cuda()], dy[rows.cuda()]
    want_y, _ = R.ffn_forward(xs, w, spec, sub, None)
    R.check(y[rows.cuda()], want_y, "y")
    # their rows of pre (the pass's own input): sorted position of each of their slots
    at = torch.empty(T * 8, dtype=torch.long)
    at[routing[1].cpu().long()] = torch.arange(T * 8)
    slots = sub[1].cpu().long()
    pre_s = pre[at[rows[slots // 8] * 8 + slots % 8].cuda()]
    want = R.ffn_backward(dys, xs, w, pre_s, spec, sub)
    R.check(got["x"][rows.cuda()], want["x"], "x")
    R.check(got["topk_w"][rows.cuda()], want["topk_w"], "topk_w")
    for n in ("gate_w", "up_w", "down_w"):
        R.check(got[n], want[n], n)
    rest = torch.ones(T, dtype=torch.bool)
    rest[rows] = False
    assert not y[rest.cuda()].any() and not got["x"][rest.cuda()].any()


def test_offsets_past_32_bits():
    """Rows whose element offsets pass 2^31: norm and linear on a [T, H] of 2.2 G elements."""
    T, H = 300_000, 7168
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    g = gen(51)
    rows = torch.tensor([0, 149_797, 299_592, 299_999], device="cuda")  # 299593 * 7168 > 2^31
    part = rand(g, (4, H), "bf16")
    x[rows] = part
    w = rand(g, (H,), "bf16", 0.3, 1.0)
    norm = train.Norm(H)
    y, stats = norm.forward(x, w)
    R.check(y[rows], R.norm_forward(part, w, None, 1e-6, "rms")[0], "norm rows")
    del y
    lin = train.Linear(H, 64)
    lw = rand(g, (64, H), "bf16", H ** -0.5)
    out = lin.forward(x, lw)
    R.check(out[rows], R.linear_forward(part, lw, None, None, "none")[0], "linear rows")
    dy = torch.zeros((T, 64), dtype=torch.bfloat16, device="cuda")
    dy[rows] = rand(g, (4, 64), "bf16")
    dx, dw, _ = lin.backward(dy, x, lw, bias_grad=False)
    want = R.linear_backward(dy[rows], part, lw, None, "none")
    R.check(dx[rows], want[0], "dx rows")
    R.check(dw, want[1], "dw")
    ok(lin)
