"""include/moe_train.h on the host (no GPU): exports, struct layout, refusals."""
import ctypes
import os
import re
import subprocess

import pytest

from sparse_moe_ffn_gemv_b200 import build, inputs
from sparse_moe_ffn_gemv_b200 import moe as M
from sparse_moe_ffn_gemv_b200 import train

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_train.h")
PTR = 0x10000  # aligned and never followed: every call below fails before it launches
INVALID, OVERFLOW, MISSING = (M.STATUS_CODE[s] for s in
                              ("MOE_ERR_INVALID_ARGUMENT", "MOE_ERR_SHAPE_OVERFLOW", "MOE_ERR_MISSING_TENSOR"))
UNSUPPORTED, SMALL = M.STATUS_CODE["MOE_ERR_UNSUPPORTED"], M.STATUS_CODE["MOE_ERR_WORKSPACE_TOO_SMALL"]


@pytest.fixture(scope="module", autouse=True)
def built_library():
    build.build()
    yield


def test_library_exports_every_declared_symbol():
    names = sorted(set(re.findall(r"MOE_API\s+moe_status\s+(moe_\w+)\s*\(", open(HEADER).read())))
    assert sorted(train.EXPORTS) == names
    out = subprocess.run(["nm", "-D", "--defined-only", M.LIB_PATH], capture_output=True, text=True).stdout
    assert set(names) <= set(re.findall(r" T (moe_\w+)", out))


def test_struct_layout_matches_the_header(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe_train.h"\nint main(void){\n'
                   'printf("%zu %zu %zu %zu %zu\\n", sizeof(moe_linear_desc), sizeof(moe_norm_desc),'
                   ' sizeof(moe_ffn_grads), offsetof(moe_norm_desc, eps), offsetof(moe_ffn_grads, down_b));'
                   'return 0;}\n')
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = list(map(int, subprocess.check_output([str(exe)]).split()))
    assert got == [ctypes.sizeof(train.MoeLinearDesc), ctypes.sizeof(train.MoeNormDesc),
                   ctypes.sizeof(train.MoeFfnGrads), train.MoeNormDesc.eps.offset, train.MoeFfnGrads.down_b.offset]


def size(fn, desc, T, backward):
    out = ctypes.c_size_t(123)
    return getattr(train.lib(), fn)(ctypes.byref(desc), T, backward, ctypes.byref(out)), out.value


@pytest.mark.parametrize("fields,T,status", [
    ((64, 128, 0, 1), 10, 0), ((64, 128, 2, 0), 0, 0), ((4, 12, 1, 0), 5, 0),
    ((0, 128, 0, 1), 10, INVALID), ((64, -8, 0, 1), 10, INVALID), ((64, 128, 3, 1), 10, INVALID),
    ((64, 128, -1, 1), 10, INVALID), ((64, 128, 0, 2), 10, INVALID), ((64, 128, 0, 3), 10, INVALID),
    ((60, 128, 0, 1), 10, INVALID), ((64, 124, 0, 1), 10, INVALID), ((66, 128, 0, 0), 10, INVALID),
    ((64, 128, 0, 1), -1, INVALID), ((64, 128, 0, 1), 2 ** 31, OVERFLOW), ((2 ** 20, 8, 0, 1), 2 ** 29, OVERFLOW),
])
def test_linear_shapes(fields, T, status):
    got, n = size("moe_linear_workspace_size", train.MoeLinearDesc(*fields), T, 1)
    assert got == status
    assert (n == 123) == (status != 0)  # written on success only


@pytest.mark.parametrize("fields,T,status", [
    ((64, 0, 1, 1e-6), 10, 0), ((20008, 1, 1, 1e-6), 1, 0), ((4, 0, 0, 1e-6), 0, 0),
    ((0, 0, 1, 1e-6), 10, INVALID), ((64, 2, 1, 1e-6), 10, INVALID), ((64, 0, 2, 1e-6), 10, INVALID),
    ((60, 0, 1, 1e-6), 10, INVALID), ((64, 0, 1, 0.0), 10, INVALID), ((64, 0, 1, float("nan")), 10, INVALID),
    ((64, 0, 1, float("inf")), 10, INVALID), ((64, 0, 1, -1.0), 10, INVALID), ((64, 0, 1, 1e-6), -5, INVALID),
    ((2 ** 20, 0, 1, 1e-6), 2 ** 29, OVERFLOW),
])
def test_norm_shapes(fields, T, status):
    assert size("moe_norm_workspace_size", train.MoeNormDesc(*fields), T, 1)[0] == status


SPEC = inputs.MoeSpec(name="t", config_id=0, hidden=64, num_experts=4, top_k=2, intermediate=32)


@pytest.mark.parametrize("spec,T,status", [
    (SPEC, 10, 0), (SPEC.replace(act_dtype="f32", weight_format="f32"), 10, 0), (SPEC, 0, 0),
    (SPEC.replace(hidden=256, intermediate=64, weight_format="q4", group_size=64), 10, UNSUPPORTED),
    (SPEC.replace(weight_format="mxfp4", intermediate=64, group_size=32), 10, UNSUPPORTED),
    (SPEC.replace(top_k=5), 10, INVALID), (SPEC.replace(hidden=60), 10, INVALID), (SPEC, -1, INVALID),
    (SPEC, 2 ** 30, OVERFLOW), (SPEC.replace(hidden=2 ** 20), 2 ** 28, OVERFLOW),
])
def test_ffn_shapes(spec, T, status):
    cfg = M.config_from_spec(spec)
    for backward in (0, 1):
        assert size("moe_ffn_workspace_size", cfg, T, backward)[0] == status


def linear_forward(d=None, **kw):
    a = dict(x=PTR, ldx=64, w=PTR, bias=None, residual=None, ldr=0, T=10, y=PTR, ldy=128, pre=None, ws=None, n=0,
             status=None)
    a.update(kw)
    return train.lib().moe_linear_forward(ctypes.byref(d or train.MoeLinearDesc(64, 128, 0, 1)), *a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(w=None), dict(y=None), dict(x=PTR + 8), dict(w=PTR + 2), dict(y=PTR + 4), dict(bias=PTR + 2),
    dict(residual=PTR, ldr=120), dict(residual=PTR, ldr=132), dict(residual=PTR + 8, ldr=128), dict(pre=PTR + 1),
    dict(ldx=56), dict(ldx=68), dict(ldy=127), dict(ldy=0), dict(ldx=-64), dict(status=PTR + 2), dict(T=-1),
])
def test_linear_forward_refusals(kw):
    assert linear_forward(**kw) == INVALID
    assert linear_forward(T=0, **{k: v for k, v in kw.items() if k != "T"}) == 0  # nothing to read or write


def linear_backward(act=0, **kw):
    a = dict(dy=PTR, lddy=128, x=PTR, ldx=64, w=PTR, pre=None, T=10, dx=PTR, lddx=64, dw=PTR, db=PTR, ws=PTR,
             n=1 << 30, status=None)
    a.update(kw)
    return train.lib().moe_linear_backward(ctypes.byref(train.MoeLinearDesc(64, 128, act, 1)), *a.values(), None)


@pytest.mark.parametrize("act,kw,status", [
    (0, dict(dy=None), INVALID), (0, dict(x=None), INVALID), (0, dict(w=None), INVALID), (1, dict(), MISSING),
    (1, dict(pre=PTR + 4), INVALID), (0, dict(lddy=120), INVALID), (0, dict(ldx=4), INVALID),
    (0, dict(lddx=66), INVALID), (0, dict(dx=PTR + 2), INVALID), (0, dict(dw=PTR + 2), INVALID),
    (0, dict(db=PTR + 2), INVALID), (0, dict(ws=None), INVALID), (0, dict(n=16), SMALL),
    (2, dict(pre=PTR, n=16), SMALL),
])
def test_linear_backward_refusals(act, kw, status):
    assert linear_backward(act, **kw) == status


def weights(cls=None, **kw):
    w = (cls or M.MoeWeights)()
    for f in ("gate_w", "up_w", "down_w"):
        setattr(w, f, PTR)
    for f, v in kw.items():
        setattr(w, f, v)
    return w


def ffn_forward(spec=SPEC, w=None, **kw):
    a = dict(u=PTR, ldu=64, T=10, off=PTR, slots=PTR, wts=PTR, residual=None, ldr=0, y=PTR, ldy=64, pre=PTR, ws=PTR,
             n=1 << 30, status=None)
    a.update(kw)
    return train.lib().moe_ffn_forward(ctypes.byref(M.config_from_spec(spec)), ctypes.byref(w or weights()),
                                       *a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(u=None), INVALID), (dict(y=None), INVALID), (dict(ldu=60), INVALID), (dict(ldy=68), INVALID),
    (dict(pre=PTR + 2), INVALID), (dict(off=None), INVALID), (dict(slots=None), INVALID), (dict(wts=None), INVALID),
    (dict(off=None, slots=None, wts=None), INVALID),   # four experts need a routing
    (dict(residual=PTR, ldr=8), INVALID), (dict(ws=None), INVALID), (dict(n=64), SMALL), (dict(T=-3), INVALID),
    (dict(T=2 ** 30), OVERFLOW), (dict(w=weights(up_w=None)), MISSING), (dict(w=weights(down_w=None)), MISSING),
    (dict(w=weights(gate_w=PTR + 8)), INVALID),
    (dict(spec=SPEC.replace(has_expert_bias=True)), MISSING),
    (dict(spec=SPEC.replace(gate_up_interleaved=True)), MISSING),
    (dict(spec=SPEC.replace(has_expert_bias=True), w=weights(gate_b=PTR, up_b=PTR)), MISSING),
    (dict(spec=SPEC.replace(weight_format="mxfp4", intermediate=64, group_size=32)), UNSUPPORTED),
])
def test_ffn_forward_refusals(kw, status):
    assert ffn_forward(**kw) == status


def ffn_backward(spec=SPEC, w=None, g=None, **kw):
    a = dict(u=PTR, ldu=64, T=10, off=PTR, slots=PTR, wts=PTR, pre=PTR, dy=PTR, lddy=64, du=PTR, lddu=64, dwt=PTR)
    b = dict(ws=PTR, n=1 << 30, status=None)
    a.update({k: v for k, v in kw.items() if k in a})
    b.update({k: v for k, v in kw.items() if k in b})
    grads = g or weights(train.MoeFfnGrads)
    return train.lib().moe_ffn_backward(ctypes.byref(M.config_from_spec(spec)), ctypes.byref(w or weights()),
                                        *a.values(), ctypes.byref(grads), *b.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(u=None), INVALID), (dict(dy=None), INVALID), (dict(pre=None), INVALID), (dict(lddy=4), INVALID),
    (dict(lddu=60), INVALID), (dict(du=PTR + 2), INVALID), (dict(dwt=PTR + 2), INVALID), (dict(n=64), SMALL),
    (dict(g=weights(train.MoeFfnGrads, down_w=None)), MISSING),
    (dict(g=weights(train.MoeFfnGrads, gate_w=PTR + 4)), INVALID),
    (dict(spec=SPEC.replace(num_experts=1, top_k=1), off=None, slots=None, wts=None), INVALID),  # dtopk_w of a dense FFN
    (dict(spec=SPEC.replace(has_expert_bias=True), w=weights(gate_b=PTR, up_b=PTR, down_b=PTR)), MISSING),
])
def test_ffn_backward_refusals(kw, status):
    assert ffn_backward(**kw) == status


@pytest.mark.parametrize("kind,kw,status", [
    (0, dict(x=None), INVALID), (0, dict(w=None), INVALID), (0, dict(y=None), INVALID), (1, dict(b=PTR), INVALID),
    (0, dict(b=PTR + 2), INVALID), (0, dict(ldx=60), INVALID), (0, dict(ldy=65), INVALID),
    (0, dict(stats=PTR + 4), INVALID), (0, dict(T=-1), INVALID),
])
def test_norm_forward_refusals(kind, kw, status):
    a = dict(x=PTR, ldx=64, w=PTR, b=None, T=10, y=PTR, ldy=64, stats=None)
    a.update(kw)
    d = train.MoeNormDesc(64, kind, 1, 1e-6)
    assert train.lib().moe_norm_forward(ctypes.byref(d), *a.values(), None) == status


@pytest.mark.parametrize("kind,kw,status", [
    (0, dict(dy=None), INVALID), (0, dict(x=None), INVALID), (0, dict(w=None), INVALID), (0, dict(stats=None), INVALID),
    (1, dict(db=PTR), INVALID), (0, dict(lddx=60), INVALID), (0, dict(lddy=12), INVALID), (0, dict(n=16), SMALL),
    (0, dict(ws=None), INVALID), (0, dict(dw=PTR + 2), INVALID),
])
def test_norm_backward_refusals(kind, kw, status):
    a = dict(dy=PTR, lddy=64, x=PTR, ldx=64, w=PTR, stats=PTR, T=10, dx=PTR, lddx=64, dw=PTR, db=None, ws=PTR,
             n=1 << 30)
    a.update(kw)
    d = train.MoeNormDesc(64, kind, 1, 1e-6)
    assert train.lib().moe_norm_backward(ctypes.byref(d), *a.values(), None) == status


FAR = 1 << 30  # from one tensor to the next: nothing overlaps


@pytest.mark.parametrize("y,kw", [
    (PTR, dict()), (PTR + 16, dict()), (PTR - 16, dict()), (PTR + 9 * 128, dict()),  # x's own, shifted, its last row
    (PTR + 112, dict(ldx=200, ldy=200)), (PTR + 128, dict(ldx=136, ldy=136)),        # side by side, but not quite
    (PTR + 128, dict(ldx=256, ldy=128)),                                             # other strides: not told apart
])
def test_linear_output_over_its_input(y, kw):
    assert linear_forward(w=FAR, y=y, **kw) == INVALID


@pytest.mark.parametrize("residual,ldr", [(2 * FAR + 16, 128), (2 * FAR, 136), (2 * FAR - 256, 128)])
def test_outputs_over_a_shifted_residual(residual, ldr):
    assert linear_forward(w=FAR, y=2 * FAR, residual=residual, ldr=ldr) == INVALID
    assert ffn_forward(y=2 * FAR, ldy=128, residual=residual, ldr=ldr) == INVALID


def test_input_gradients_over_inputs():
    assert linear_backward(dx=PTR, dy=FAR) == INVALID            # x's
    assert linear_backward(dx=PTR, x=FAR) == INVALID             # dy's
    assert ffn_backward(du=PTR, dy=FAR) == INVALID
    assert ffn_backward(du=PTR, u=FAR) == INVALID
    assert ffn_forward(u=PTR, y=PTR + 128) == INVALID            # u itself would be right, its next row is not
    d = train.MoeNormDesc(64, 0, 1, 1e-6)
    norm = train.lib().moe_norm_backward
    for dy, x in ((PTR, FAR), (FAR, PTR)):
        assert norm(ctypes.byref(d), dy, 64, x, 64, PTR, PTR, 10, PTR, 64, None, None, PTR, 1 << 30, None) == INVALID
    fwd = train.lib().moe_norm_forward
    assert fwd(ctypes.byref(d), PTR, 64, PTR, None, 10, PTR + 128, 64, None, None) == INVALID
    assert fwd(ctypes.byref(d), PTR, 64, PTR, None, 10, PTR, 72, None, None) == INVALID


def test_widths_past_their_limit():
    wide = 1 << 28
    assert size("moe_linear_workspace_size", train.MoeLinearDesc(wide + 8, 8, 0, 1), 1, 0)[0] == OVERFLOW
    assert size("moe_linear_workspace_size", train.MoeLinearDesc(8, wide + 8, 0, 1), 1, 0)[0] == OVERFLOW
    assert size("moe_linear_workspace_size", train.MoeLinearDesc(8, wide, 0, 1), 1, 1)[0] == 0
    assert size("moe_norm_workspace_size", train.MoeNormDesc(wide + 8, 0, 1, 1e-6), 1, 0)[0] == OVERFLOW
    one = SPEC.replace(num_experts=1, top_k=1, hidden=8)
    assert size("moe_ffn_workspace_size", M.config_from_spec(one.replace(intermediate=wide + 8)), 1, 0)[0] == OVERFLOW
    assert size("moe_ffn_workspace_size", M.config_from_spec(one.replace(intermediate=wide)), 1, 1)[0] == 0
