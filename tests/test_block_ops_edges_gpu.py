"""Residual norms and rotary positions where the other tests do not go."""
import math

import pytest
import torch

import block_ops_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,r,H,T", [(128, 128, 1, 7), (6, 6, 3, 7), (128, 128, 40, 2048), (66, 66, 24, 8192)])
def test_sine_of_a_small_angle(cuda_lib, d, r, H, T, interleaved):
    """The pair (0, 1) turns to (-sin, cos), each within 8 roundings of itself however small the angle, and 2^-55 turn:
    the angle's two words are rounded, their sum, the constant, the product with it (4); the polynomial adds its last
    step and, its terms being a tenth of the angle at most, half a rounding in all (1.5); its remainder is below 2.3e-9
    of the sine (0.04); the factor, 1, and the product with 1 are exact.  Short calls and long ones, vectors and
    single elements."""
    plan = cuda_lib.foak_rotary_plan(r, base=1e7, interleaved=interleaved, scaling="linear", factor=8.0)
    pos = torch.tensor([1, -1, 2, 3, -100, 2 ** 20 + 1, 0])[torch.arange(T) % 7]
    x = torch.zeros(T, H, d)
    half = torch.arange(r // 2)
    first, second = (2 * half, 2 * half + 1) if interleaved else (half, half + r // 2)
    x[:, :, second] = 1.0
    out = cuda_lib.foak_rotary_apply(plan, pos.cuda(), x.cuda())[0].cpu()
    assert torch.equal(out[7:], out[:-7]) and torch.equal(out[:, 1:], out[:, :-1])
    for t in range(7):
        for i, turn in enumerate(plan.turns.tolist()):
            whole = int(pos[t]) * turn % 2 ** 64
            angle = (whole - 2 ** 64 if whole >= 2 ** 63 else whole) / 2.0 ** 64 * (2.0 * math.pi)
            for got, want in ((out[t, 0, first[i]], -math.sin(angle)), (out[t, 0, second[i]], math.cos(angle))):
                assert abs(float(got) - want) <= 8 * ref.U * abs(want) + 2 * math.pi * 2.0 ** -55, (int(pos[t]), i, float(got), want)
