"""The training operators on the GPU where their kernels change form: rings that wrap, sums of many
rows, problems past a threshold (tests/train_ref.py has the 64-bit definitions)."""
import ctypes

import pytest
import torch

import train_ref as R
from sparse_moe_ffn_gemv_b200 import train
from test_train_ops import ffn_case, gen, ok, padded, rand, spec_of

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("dtype,T,H,kind,pad", [
    # a block's ring of 8, 3 and 2 stages goes round; the last row group is not full
    ("bf16", 40_003, 64, "layer", 8), ("bf16", 20_001, 136, "rms", 0), ("bf16", 2_000, 7168, "layer", 8),
    ("bf16", 1_200, 8192, "rms", 0), ("f32", 1_301, 4096, "layer", 4), ("f32", 9_001, 516, "rms", 0),
    ("bf16", 297, 7168, "rms", 0), ("bf16", 9, 264, "layer", 0),
])
def test_norm_backward_over_many_rows(dtype, T, H, kind, pad):
    g = gen(T + 3 * H)
    x, dy = padded(g, T, H, pad, dtype, 2.0), padded(g, T, H, pad, dtype)
    w = rand(g, (H,), dtype, 0.3, 1.0)
    op = train.Norm(H, kind=kind, eps=1e-5, dtype=dtype)
    _, stats = op.forward(x, w)
    dx, dw, db = op.backward(dy, x, w, stats)
    ok(op)
    want = R.norm_backward(dy, x, w, stats, kind)
    R.check(dx, want[0], "dx")
    R.check(dw, want[1], "dw")
    if kind == "layer":
        R.check(db, want[2], "db")
    again = op.backward(dy, x, w, stats)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    assert torch.equal(op.backward(dy, x, w, stats, input_grad=False)[1], dw)


# ------------------------------------------------------------------ f32 products past a threshold
@pytest.mark.parametrize("T,K,N,act", [(1200, 768, 768, "silu"), (1201, 772, 764, "none"), (2600, 516, 1028, "gelu")])
def test_f32_gradients_do_not_depend_on_the_others(T, K, N, act):
    """Sizes at which the products of the pass together, but not each alone, take the form of large
    problems: a gradient asked for alone has the same bits."""
    g = gen(T + K)
    x, w, dy = rand(g, (T, K), "f32"), rand(g, (N, K), "f32", K ** -0.5), rand(g, (T, N), "f32")
    pre = rand(g, (T, N), "f32", 1.5) if act != "none" else None
    op = train.Linear(K, N, activation=act, dtype="f32")
    dx, dw, db = op.backward(dy, x, w, pre=pre)
    want = R.linear_backward(dy, x, w, pre, act)
    for got, ref, name in zip((dx, dw, db), want, ("dx", "dw", "db")):
        R.check(got, ref, name)
    for kw in (dict(input_grad=False), dict(weight_grad=False), dict(bias_grad=False), dict(input_grad=False, bias_grad=False),
               dict(weight_grad=False, bias_grad=False), dict(input_grad=False, weight_grad=False)):
        for alone, got in zip(op.backward(dy, x, w, pre=pre, **kw), (dx, dw, db)):
            assert alone is None or torch.equal(alone, got)
    ok(op)


@pytest.mark.parametrize("T,kw", [
    (2000, dict(hidden=388, intermediate=260)), (1300, dict(num_experts=3, top_k=2, hidden=260, intermediate=132, has_expert_bias=True)),
])
def test_f32_ffn_weight_gradients_do_not_depend_on_the_input_gradient(T, kw):
    spec, g, w, routing = ffn_case(T, None, dict(kw, act_dtype="f32"))
    x, dy = (rand(g, (T, spec.hidden), "f32") for _ in range(2))
    pre = rand(g, (T * spec.top_k, 2 * spec.intermediate), "f32", 1.2)
    op = train.GatedFfn(spec)
    got = op.backward(dy, x, w, pre, routing=routing)
    less = op.backward(dy, x, w, pre, routing=routing, input_grad=False)
    ok(op)
    assert set(got) - set(less) == {"x"}
    for n in less:
        assert torch.equal(less[n], got[n]), n


LARGE_F32 = [  # at least 296 tiles of 64 x 64 in each product, with remainders
    (2100, None, dict(hidden=580, intermediate=324)),
    (2101, None, dict(hidden=580, intermediate=324, gate_up_interleaved=True, has_expert_bias=True,
                      activation="swiglu_clamped", swiglu_limit=1.0)),
    (900, 44, dict(num_experts=46, top_k=4, hidden=324, intermediate=164, has_expert_bias=True)),
]


@pytest.mark.parametrize("T,K,N", [(1501, 772, 836), (4099, 36, 324), (330, 2500, 4100)])
def test_large_f32_linear(T, K, N):
    g = gen(T + K)
    x, w, b = padded(g, T, K, 4, "f32"), rand(g, (N, K), "f32", K ** -0.5), rand(g, (N,), "f32", 0.3)
    r, dy = padded(g, T, N, 8, "f32"), padded(g, T, N, 4, "f32")
    op = train.Linear(K, N, activation="silu", dtype="f32")
    y, pre = op.forward(x, w, bias=b, residual=r, keep=True)
    want_y, want_z = R.linear_forward(x, w, b, r, "silu")
    R.check(y, want_y, "y")
    R.check(pre, want_z, "pre")
    want = R.linear_backward(dy, x, w, pre, "silu")
    for got, ref, name in zip(op.backward(dy, x, w, pre=pre), want, ("dx", "dw", "db")):
        R.check(got, ref, name)
    ok(op)


@pytest.mark.parametrize("T,experts,kw", LARGE_F32)
def test_large_f32_ffn(T, experts, kw):
    spec, g, w, routing = ffn_case(T, experts, dict(kw, act_dtype="f32"))
    x, dy = (padded(g, T, spec.hidden, 4, "f32") for _ in range(2))
    op = train.GatedFfn(spec)
    y, pre = op.forward(x, w, routing=routing)
    want_y, want_pre = R.ffn_forward(x, w, spec, routing, None)
    R.check(pre, want_pre, "pre")
    R.check(y, want_y, "y")
    got = op.backward(dy, x, w, pre, routing=routing)
    ok(op)
    want = R.ffn_backward(dy, x, w, pre, spec, routing)
    assert set(got) == set(want)
    for name in want:
        R.check(got[name], want[name], name)


def test_ffn_bias_gradients_of_very_wide_planes():
    """2^24 gate and up columns: more blocks of column sums than a launch has in its second
    dimension."""
    spec = spec_of(hidden=8, intermediate=1 << 23, act_dtype="f32", has_expert_bias=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    new = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    I = spec.intermediate
    w = {"gate_w": new(1, I, 8), "up_w": new(1, I, 8), "down_w": new(1, 8, I), "gate_b": new(1, I), "up_b": new(1, I),
         "down_b": new(1, 8)}
    x, dy, pre = new(3, 8), new(3, 8), new(3, 2 * I)
    op = train.GatedFfn(spec)
    got = op.backward(dy, x, w, pre, input_grad=False)
    ok(op)
    want = R.ffn_backward(dy, x, w, pre, spec, None)
    for n in ("gate_b", "up_b", "down_b", "gate_w", "down_w"):
        R.check(got[n], want[n], n)


# ------------------------------------------------------------------ workspace of the dense FFN
@pytest.mark.parametrize("T,kw", [(2, dict(hidden=512, intermediate=512)), (1500, dict(hidden=2048, intermediate=512)),
                                  (700, dict(hidden=1024, intermediate=264, has_expert_bias=True)),
                                  (300, dict(hidden=516, intermediate=260, act_dtype="f32", has_expert_bias=True))])
def test_dense_ffn_takes_no_second_copy_of_its_rows(T, kw):
    """What a call allocates beside its results: the hidden rows and the sums' partial rows."""
    spec, g, w, _ = ffn_case(T, None, kw)
    x, dy = rand(g, (T, spec.hidden), spec.act_dtype), rand(g, (T, spec.hidden), spec.act_dtype)
    op = train.GatedFfn(spec)
    y, pre = op.forward(x, w)
    want = op.backward(dy, x, w, pre)
    ok(op)
    I, H, es = spec.intermediate, spec.hidden, x.element_size()
    partial = -(-T // 128) * (2 * I + H) * 4 if spec.has_expert_bias else 0
    room = 3 << 20  # blocks of the allocator are rounded up
    for call, most in ((lambda: op.forward(x, w, keep=False)[0], T * H * es + T * I * es * (5 if es == 4 else 1)),
                       (lambda: list(op.backward(dy, x, w, pre).values()),
                        sum(t.numel() * es for t in want.values()) + T * I * es * (4 if es == 4 else 3) + partial)):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        out = call()
        used = torch.cuda.max_memory_allocated() - before
        assert used <= most + room, (used, most)
        del out


@pytest.mark.parametrize("kw", [dict(hidden=264, intermediate=200, has_expert_bias=True),
                                dict(hidden=132, intermediate=68, act_dtype="f32", has_expert_bias=True)])
@pytest.mark.parametrize("T", [1, 3, 5, 129, 1000])
def test_dense_ffn_stays_in_its_workspace(T, kw):
    """The C calls with a workspace of exactly the size asked for, which lies between marked bytes."""
    spec, g, w, _ = ffn_case(T, None, kw)
    dt = x_dt = spec.act_dtype
    x, dy = rand(g, (T, spec.hidden), x_dt), rand(g, (T, spec.hidden), dt)
    op = train.GatedFfn(spec)
    y, pre = op.forward(x, w)
    want = op.backward(dy, x, w, pre)
    lib, p = op.lib, lambda t: t.data_ptr()  # noqa: E731
    stream = torch.cuda.current_stream().cuda_stream
    for backward in (0, 1):
        n = ctypes.c_size_t()
        assert lib.moe_ffn_dense_workspace_size(op._cfg, T, backward, ctypes.byref(n)) == 0
        room = torch.full((n.value + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        ws = p(room) + 4096
        if backward:
            got = {k: torch.empty_like(v) for k, v in want.items()}
            grads = train.MoeFfnGrads(**{k: p(v) for k, v in got.items() if k != "x"})
            assert lib.moe_ffn_backward(op._cfg, ctypes.byref(op._planes(w)), p(x), spec.hidden, T, None, None, None, p(pre),
                                        p(dy), spec.hidden, p(got["x"]), spec.hidden, None, ctypes.byref(grads), ws, n.value,
                                        p(op.status), stream) == 0
            assert all(torch.equal(got[k], want[k]) for k in want)
        else:
            out = torch.empty_like(y)
            assert lib.moe_ffn_forward(op._cfg, ctypes.byref(op._planes(w)), p(x), spec.hidden, T, None, None, None, None, 0,
                                       p(out), spec.hidden, None, ws, n.value, p(op.status), stream) == 0
            assert torch.equal(out, y)
        ok(op)
        assert (room[:4096] == 0xA5).all() and (room[4096 + n.value:] == 0xA5).all()
