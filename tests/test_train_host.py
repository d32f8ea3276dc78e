"""include/moe_train.h on the host (no GPU): sizes past the limits, what an import needs."""
import ctypes
import os
import subprocess
import sys

import pytest

from sparse_moe_ffn_gemv_b200 import build, inputs
from sparse_moe_ffn_gemv_b200 import moe as M
from sparse_moe_ffn_gemv_b200 import train

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OVERFLOW = M.STATUS_CODE["MOE_ERR_SHAPE_OVERFLOW"]


@pytest.fixture(scope="module", autouse=True)
def built_library():
    build.build()
    yield


def size(fn, desc, T, backward):
    out = ctypes.c_size_t(123)
    return getattr(train.lib(), fn)(ctypes.byref(desc), T, backward, ctypes.byref(out))


@pytest.mark.parametrize("fields,T,status", [
    ((1 << 24, 1 << 24, 0, 1), 1, OVERFLOW),           # a weight plane of 2^48 elements
    ((1 << 24, 1 << 24, 0, 0), 0, OVERFLOW),
    ((1 << 23, 1 << 23, 0, 0), 1, OVERFLOW),           # 2^46 elements: 2^34 tiles of f32
    ((8, 1 << 28, 0, 1), 1 << 18, OVERFLOW),           # 2^31 tiles of the forward product,
    ((1 << 28, 8, 0, 1), 1 << 18, OVERFLOW),           # of the input gradient
    ((8, 1 << 28, 0, 1), 1 << 15, 0), ((8, 1 << 28, 0, 0), 1 << 12, 0),
    ((1 << 18, 1 << 18, 0, 1), 16, 0),                 # 137 GB of weights
])
def test_linear_planes_and_tiles(fields, T, status):
    for backward in (0, 1):
        assert size("moe_linear_workspace_size", train.MoeLinearDesc(*fields), T, backward) == status


@pytest.mark.parametrize("kw,T,status", [
    (dict(hidden=1 << 17, intermediate=1 << 19, num_experts=512), 1, OVERFLOW),     # planes of 2^46 elements
    (dict(hidden=1 << 14, intermediate=1 << 21, num_experts=512), 1, OVERFLOW),     # 2^45: 2^30 tiles of a weight gradient
    (dict(hidden=8, intermediate=1 << 27, num_experts=1, top_k=1), 1 << 18, OVERFLOW),  # 2^31 tiles of gate and up
    (dict(hidden=1 << 12, intermediate=1 << 12, num_experts=512), 1 << 14, 0),
])
def test_ffn_planes_and_tiles(kw, T, status):
    spec = inputs.MoeSpec(**{**dict(name="t", config_id=0, num_experts=4, top_k=2), **kw})
    for backward in (0, 1):
        assert size("moe_ffn_workspace_size", M.config_from_spec(spec), T, backward) == status


def test_import_without_cuda_in_torch():
    """A PyTorch built without CUDA lacks the runtime's functions: the module imports, the size calls
    work, and a handle raises."""
    prog = """
import torch
for n in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, n)
import ctypes
from sparse_moe_ffn_gemv_b200 import train
n = ctypes.c_size_t()
assert train.lib().moe_linear_workspace_size(ctypes.byref(train.MoeLinearDesc(64, 64, 1, 1)), 5, 1, ctypes.byref(n)) == 0
for make in (lambda: train.Linear(64, 64), lambda: train.Norm(64, device="cuda:0")):
    try:
        make()
    except (RuntimeError, AssertionError, AttributeError) as e:
        print("raised", type(e).__name__)
"""
    run = subprocess.run([sys.executable, "-c", prog], cwd=ROOT, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
    assert run.stdout.count("raised") == 2


def dense_size(spec, T, backward):
    out = ctypes.c_size_t(123)
    fn = train.lib().moe_ffn_dense_workspace_size
    return fn(ctypes.byref(M.config_from_spec(spec)), T, backward, ctypes.byref(out)), out.value


ONE = inputs.MoeSpec(name="t", config_id=0, hidden=7168, num_experts=1, top_k=1, intermediate=2048)


@pytest.mark.parametrize("spec", [ONE, ONE.replace(has_expert_bias=True), ONE.replace(act_dtype="f32", weight_format="f32")])
def test_dense_ffn_workspace(spec):
    """h forward; dg, dv, w h (and the f32 dh) and the bias gradients' partial sums backward, each
    rounded up to 256 bytes: no copy of the rows."""
    I, es = spec.intermediate, 4 if spec.act_dtype == "f32" else 2
    for T in (0, 1, 300, 8192):
        status, fwd = dense_size(spec, T, 0)
        assert status == 0 and fwd <= T * I * es * (5 if es == 4 else 1) + 512
        status, back = dense_size(spec, T, 1)
        partial = -(-T // 128) * (2 * I + spec.hidden) * 4 if spec.has_expert_bias else 0
        assert status == 0 and back <= T * I * es * (4 if es == 4 else 3) + partial + 1024
        out = ctypes.c_size_t()
        assert train.lib().moe_ffn_workspace_size(ctypes.byref(M.config_from_spec(spec)), T, 1, ctypes.byref(out)) == 0
        assert out.value >= back
    invalid = M.STATUS_CODE["MOE_ERR_INVALID_ARGUMENT"]
    assert dense_size(spec.replace(num_experts=4), 10, 0)[0] == invalid
    assert dense_size(spec, -1, 0) == (invalid, 123)


@pytest.mark.parametrize("make,name", [
    (lambda n: train.Linear(n, 64), "in_features"), (lambda n: train.Linear(64, n), "out_features"),
    (lambda n: train.Norm(n), "width"), (lambda n: train.GatedFfn(ONE.replace(hidden=n)), "hidden"),
    (lambda n: train.GatedFfn(ONE.replace(intermediate=n)), "intermediate"),
])
def test_sizes_that_a_c_int_does_not_hold(make, name):
    """2^32 + 64 is not 64: refused before anything else is asked of the device."""
    for n in (2 ** 32 + 64, 2 ** 31, -2 ** 31 - 8):
        with pytest.raises(M.MoeError, match=name) as e:
            make(n)
        assert e.value.name == "MOE_ERR_SHAPE_OVERFLOW"
