"""The training operators on the GPU where their kernels change form: rings that wrap, sums of many
rows, problems past a threshold (tests/train_ref.py has the 64-bit definitions)."""
import pytest
import torch

import train_ref as R
from sparse_moe_ffn_gemv_b200 import train
from test_train_ops import padded, rand, gen, ok

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
