"""GPU parity of rotary positions: layouts, parts of the head, scalings, strides, far positions."""
import pytest
import torch

import block_ops_ref as ref

pytestmark = pytest.mark.gpu


def _heads(T, H, d, dtype, seed):
    return torch.randn(T, H, d, generator=torch.Generator().manual_seed(seed)).to(ref.DT[dtype])


def _positions(T, far, seed):
    return torch.randint(0, far, (T,), generator=torch.Generator().manual_seed(seed))


def _check(ce, plan, q, k, pos, inverse=False, **given):
    turns = [t % 2 ** 64 for t in plan.turns.tolist()]
    out = ce.foak_rotary_apply(plan, pos.cuda(), None if q is None else q.cuda(), None if k is None else k.cuda(), inverse=inverse, **given)
    for x, o, name in ((q, out[0], "q"), (k, out[1], "k")):
        assert (x is None) == (o is None)
        if x is not None:
            ref.assert_close(o, ref.rotate(x, pos.tolist(), turns, plan.rotary_dim, plan.interleaved, plan.factor, inverse), name)
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,r", [(128, 128), (128, 64), (64, 32), (80, 20), (96, 24), (256, 256), (72, 8), (18, 12), (7, 6), (2, 2), (12, 4), (40, 24)])
def test_sizes(cuda_lib, d, r, interleaved, dtype):
    plan = cuda_lib.foak_rotary_plan(r, base=500000.0, interleaved=interleaved)
    for T, Hq, Hk in ((1, 1, 1), (5, 3, 2), (67, 9, 1)):
        _check(cuda_lib, plan, _heads(T, Hq, d, dtype, 1), _heads(T, Hk, d, dtype, 2), _positions(T, 8192, T))


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "bands", "ramp"])
@pytest.mark.parametrize("inverse", [False, True])
def test_scalings(cuda_lib, scaling, inverse):
    plan = cuda_lib.foak_rotary_plan(64, base=10000.0, scaling=scaling, factor=4.0, original=2048.0)
    assert (plan.factor != 1.0) == (scaling == "ramp")
    for dtype in ("bf16", "f32"):
        _check(cuda_lib, plan, _heads(33, 4, 64, dtype, 3), _heads(33, 2, 64, dtype, 4), _positions(33, 8192, 5), inverse)


def test_own_frequencies_and_factor(cuda_lib):
    plan = cuda_lib.foak_rotary_plan(6, inv_freq=[3.0, -0.25, 100.0], attention_factor=0.5, interleaved=True)
    _check(cuda_lib, plan, _heads(9, 2, 8, "f32", 3), None, _positions(9, 1000, 5))


def test_far_and_negative_positions(cuda_lib):
    """Whatever the position, the angle is a whole-number product modulo a turn."""
    plan = cuda_lib.foak_rotary_plan(128, base=500000.0)
    pos = torch.tensor([0, 1, -1, -5000, 131071, 2 ** 24 + 1, 2 ** 31 - 1, 2 ** 31, 2 ** 40 + 7, 2 ** 62, -2 ** 63])
    for dtype in ("f32", "bf16"):
        _check(cuda_lib, plan, _heads(len(pos), 3, 128, dtype, 1), _heads(len(pos), 1, 128, dtype, 2), pos)


def test_against_the_table(cuda_lib):
    """The same rotation as foak_rope_apply's, which takes cosines from a table."""
    ce = cuda_lib
    x, pos = _heads(100, 4, 128, "f32", 7).cuda(), _positions(100, 4096, 7).cuda()
    got, _ = ce.foak_rotary_apply(ce.foak_rotary_plan(128, base=10000.0), pos, x)
    ce.foak_rope_apply(x, pos, ce.foak_rope_cache(4096, 128))
    # each within 8 roundings and 4e-9 of the rotation, of elements below 6
    assert float((got - x).abs().max()) <= 2 * 12 * (8 * ref.U + 4e-9)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [128, 80, 20])
def test_strides(cuda_lib, d, dtype):
    """Parts of a fused product, heads first, places that are not 16-byte aligned; in place and out of place."""
    ce, T = cuda_lib, 41
    r = d // 4 * 2
    plan = ce.foak_rotary_plan(r, interleaved=False)
    turns = [t % 2 ** 64 for t in plan.turns.tolist()]
    pos = _positions(T, 4096, 2)
    for shift in (0, 1, 2, 8):
        flat = torch.randn(T, 11 * d + shift, generator=torch.Generator().manual_seed(shift)).to(ref.DT[dtype]).cuda()
        qkv = flat[:, shift:].unflatten(1, (11, d))
        before = flat.clone()
        q, k = qkv[:, :6], qkv[:, 6:8]
        heads_first = torch.full((8, T, d), 9.0, dtype=q.dtype, device="cuda")
        out = ce.foak_rotary_apply(plan, pos.cuda(), q, k, q_out=heads_first[:6].transpose(0, 1), k_out=heads_first[6:].transpose(0, 1))
        assert torch.equal(flat, before)
        for x, o in ((q, out[0]), (k, out[1])):
            ref.assert_close(o, ref.rotate(x, pos.tolist(), turns, r, False), "strided")
        back = ce.foak_rotary_apply(plan, pos.cuda(), heads_first.transpose(0, 1))[0]
        assert back.shape == (T, 8, d)
        ce.foak_rotary_apply(plan, pos.cuda(), q, k, q_out=q, k_out=k)  # in place
        assert torch.equal(q, out[0]) and torch.equal(k, out[1])
        assert torch.equal(flat[:, :shift], before[:, :shift]) and torch.equal(qkv[:, 8:], before[:, shift:].unflatten(1, (11, d))[:, 8:])


def test_a_head_for_all(cuda_lib):
    """An expanded input: every head of the output from the same head."""
    ce = cuda_lib
    plan = ce.foak_rotary_plan(64)
    one = _heads(12, 1, 64, "f32", 3).cuda()
    out, _ = ce.foak_rotary_apply(plan, torch.arange(12, device="cuda"), one.expand(12, 5, 64))
    alone, _ = ce.foak_rotary_apply(plan, torch.arange(12, device="cuda"), one)
    assert torch.equal(out, alone.expand(12, 5, 64))
    with pytest.raises(ce.FoakError):
        ce.foak_rotary_apply(plan, torch.arange(12, device="cuda"), out, q_out=one.expand(12, 5, 64))


@pytest.mark.parametrize("interleaved", [False, True])
def test_there_and_back(cuda_lib, interleaved):
    ce = cuda_lib
    plan = ce.foak_rotary_plan(96, interleaved=interleaved)
    x, pos = _heads(50, 3, 128, "f32", 5).cuda(), _positions(50, 10 ** 6, 5).cuda()
    y, _ = ce.foak_rotary_apply(plan, pos, x)
    z, _ = ce.foak_rotary_apply(plan, pos, y, inverse=True)
    # two rotations, 8 roundings and 4e-9 of |a| + |b| < 12 each, the second of values below 12 root 2
    assert float((z - x).abs().max()) <= 12 * 2.5 * (9 * ref.U + 4e-9)


def test_gradient_against_differences(cuda_lib):
    """The inverse is the gradient's way: a linear map's differences are exact but for roundings."""
    ce = cuda_lib
    plan = ce.foak_rotary_plan(6, interleaved=True, attention_factor=1.25)
    turns = [t % 2 ** 64 for t in plan.turns.tolist()]
    x, w, pos = _heads(3, 1, 8, "f32", 5), _heads(3, 1, 8, "f32", 6), [3, 100, 77777]
    grad, _ = ce.foak_rotary_apply(plan, torch.tensor(pos).cuda(), w.cuda(), inverse=True)
    base = (ref.rotate(x, pos, turns, 6, True, 1.25)[0] * w.double()).sum()
    for j in range(x.numel()):
        y = x.double()
        y.view(-1)[j] += 1.0
        slope = (ref.rotate(y, pos, turns, 6, True, 1.25)[0] * w.double()).sum() - base
        assert abs(float(grad.view(-1)[j]) - float(slope)) <= 10 * 1.25 * (8 * ref.U + 4e-9)


def test_no_tokens(cuda_lib):
    ce = cuda_lib
    plan = ce.foak_rotary_plan(64)
    q, k = ce.foak_rotary_apply(plan, torch.zeros(0, dtype=torch.int64, device="cuda"), torch.empty(0, 4, 64, device="cuda"), torch.empty(0, 2, 64, device="cuda"))
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)


def test_refusals_of_the_binding(cuda_lib):
    ce = cuda_lib
    plan, pos = ce.foak_rotary_plan(64), torch.zeros(4, dtype=torch.int64, device="cuda")
    q = torch.zeros(4, 2, 64, device="cuda")
    bad = [
        lambda: ce.foak_rotary_apply(plan, pos, None),
        lambda: ce.foak_rotary_apply(plan, pos, q[:, :, :32]),
        lambda: ce.foak_rotary_apply(plan, pos[:3], q),
        lambda: ce.foak_rotary_apply(plan, pos.int(), q),
        lambda: ce.foak_rotary_apply(plan, pos.cpu(), q),
        lambda: ce.foak_rotary_apply(plan, pos, q.half()),
        lambda: ce.foak_rotary_apply(plan, pos, q, q.bfloat16()),
        lambda: ce.foak_rotary_apply(plan, pos, q, torch.zeros(4, 2, 96, device="cuda")),
        lambda: ce.foak_rotary_apply(plan, pos, q, q_out=torch.zeros(4, 3, 64, device="cuda")),
        lambda: ce.foak_rotary_apply(plan, pos, q.transpose(1, 2)),
        lambda: ce.foak_rotary_apply(ce.foak_rotary_plan(64, device="cpu"), pos, q),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
