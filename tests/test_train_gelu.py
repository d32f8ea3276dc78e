"""GELU of a bf16 linear layer over the whole range of its argument, element by element."""
import math

import pytest
import torch

from sparse_moe_ffn_gemv_b200 import train

pytestmark = pytest.mark.gpu


def arguments():
    """Every bf16 value from -12.5 to 12.5 whose magnitude is at least 2^-10, and zero."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    z = bits.view(torch.bfloat16)
    z = z[torch.isfinite(z) & (z.abs() <= 12.5) & (z.abs() >= 2.0 ** -10)]
    return torch.cat([z, torch.zeros(1, dtype=torch.bfloat16)]).cuda()


def spread(z):
    """z as column 0 of [T, 8] rows, and the weights that hand it to every output."""
    x = torch.zeros(len(z), 8, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = z
    w = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = 1
    return x, w


def normal(z):
    """Phi in 64 bits. By erfc: torch.special.ndtr takes 1 + erf, which at -8 keeps one digit."""
    return 0.5 * torch.erfc(-z.double() / math.sqrt(2))


# the function's own error, relative: 2^-20 of the fit, the exponential's 2^-22 and the rounding of its
# argument z^2 / 2 (at most 78) times log2 e, 113 * 2^-24, on top of the result's half step
OWN = 2.0 ** -20 + 2.0 ** -22 + 113 * 2.0 ** -24 + 8 * 2.0 ** -24


@pytest.mark.parametrize("rows", [None, 1, 4])  # tensor cores, one token, few tokens
def test_gelu_is_right_to_bf16_in_its_tail(rows):
    z = arguments()
    if rows:
        z = z[torch.linspace(0, len(z) - 1, 60 * rows, device="cuda").long()]
    x, w = spread(z)
    op = train.Linear(8, 8, activation="gelu")
    y = op.forward(x, w) if rows is None else torch.cat([op.forward(x[i:i + rows], w) for i in range(0, len(z), rows)])
    want = z.double() * normal(z)
    own = OWN * want.abs() + 2.0 ** -23 * z.double().abs() * (z > 0)  # 1 - tail rounds at 1
    bound = own + 2.0 ** -8 * (want.abs() + own)
    for c in range(8):
        off = (y[:, c].double() - want).abs()
        worst = int((off - bound).argmax())
        assert not bool((off > bound).any()), (float(z[worst]), float(y[worst, c]), float(want[worst]))
    assert op.device_status() == 0


def test_gelu_derivative_is_right_to_bf16_in_its_tail():
    z = arguments()
    T = len(z)
    op = train.Linear(8, 8, activation="gelu")
    pre = z[:, None].expand(T, 8).contiguous()
    dy = torch.ones(T, 8, dtype=torch.bfloat16, device="cuda")
    eye = torch.eye(8, dtype=torch.bfloat16, device="cuda")
    x, _ = spread(z)
    dx, _, _ = op.backward(dy, x, eye, pre=pre)  # dz itself, rounded once
    z = z.double()
    Phi, slope = normal(z), z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    want = Phi + slope
    own = OWN * (Phi + slope.abs()) + 2.0 ** -23 * (z > 0)
    bound = own + 2.0 ** -8 * (want.abs() + own)
    for c in range(8):
        off = (dx[:, c].double() - want).abs()
        worst = int((off - bound).argmax())
        assert not bool((off > bound).any()), (float(z[worst]), float(dx[worst, c]), float(want[worst]))
    assert op.device_status() == 0
