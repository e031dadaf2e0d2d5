"""Residual norms and rotary positions where offsets, strides and counts pass 32 bits.  Rows of the same contents have
to give the same bits wherever they lie."""
import pytest
import torch

import block_ops_ref as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
REPEAT = 7


def _same_rows(t, what):
    """Every row equals the one REPEAT before it."""
    for a in range(0, t.shape[0] - REPEAT, 4096):
        b = min(a + 4096, t.shape[0] - REPEAT)
        assert torch.equal(t[a:b], t[a + REPEAT : b + REPEAT]), (what, a)


@pytest.mark.parametrize("post,gate", [(False, "none"), (True, "channel")])
def test_tensors_of_more_than_four_gigabytes(cuda_lib, post, gate):
    ce, N, D = cuda_lib, 70001, 32768
    c = ref.make_norm(REPEAT, D, "bf16", gate, post, seed=4)
    rows = torch.arange(N, device="cuda") % REPEAT
    big = {k: c[k].cuda()[rows] for k in ("X", "R", "dY", "dH")}
    assert big["X"].numel() * 2 > 2 ** 32
    how = dict(gate=None if c["gate"] is None else c["gate"].cuda(), post_gamma=None if not post else c["post_gamma"].cuda(), scale=0.3)
    gamma = c["gamma"].cuda()
    f = ce.foak_residual_norm_forward(big["X"], big["R"], gamma, eps=1e-5, post_eps=1e-6, H=big["R"], **how)
    want = ref.norm_forward(c["X"], c["R"], c["gamma"], c["gate"], c["post_gamma"], 0.3, 1e-5, 1e-6)
    for k in ("H", "Y", "rstd"):
        _same_rows(f[k], k)
        ref.assert_close(f[k][:REPEAT], want[k], k)
    del big["R"]
    H, Y = f["H"], f["Y"]
    b = ce.foak_residual_norm_backward(big["dY"], big["dH"], H, f["rstd"], gamma, X=big["X"], post_rstd=f["post_rstd"], dR=big["dH"], dX=Y, **how)
    seven = ref.norm_backward(c["dY"], c["dH"], H[:REPEAT], f["rstd"][:REPEAT], c["gamma"], c["X"], c["gate"], c["post_gamma"], None if not post else f["post_rstd"][:REPEAT], 0.3)
    for k in ("dR", "dX"):
        _same_rows(b[k], k)
        ref.assert_close(b[k][:REPEAT], seven[k], k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_row_strides_past_32_bits(cuda_lib, dtype):
    """Three rows, 4 GiB apart."""
    ce, N, D, dt = cuda_lib, 3, 520, ref.DT[dtype]
    ld = 2 ** 32 // dt.itemsize + 8
    c = ref.make_norm(N, D, dtype, "channel", True, seed=6)
    room = torch.empty((N - 1) * ld + D, dtype=dt, device="cuda")

    def far(t):
        v = room.as_strided((N, D), (ld, 1))
        return v if t is None else v.copy_(t)

    near = {k: None if v is None else v.cuda() for k, v in c.items()}
    how = dict(gate=near["gate"], post_gamma=near["post_gamma"], scale=0.5)
    f = ce.foak_residual_norm_forward(near["X"], near["R"], near["gamma"], **how)
    a = ce.foak_residual_norm_forward(far(c["X"]), near["R"], near["gamma"], **how)
    assert torch.equal(a["H"], f["H"]) and torch.equal(a["Y"], f["Y"])
    a = ce.foak_residual_norm_forward(near["X"], near["R"], near["gamma"], H=far(None), **how)
    assert torch.equal(a["H"], f["H"]) and torch.equal(a["Y"], f["Y"])
    want = ref.norm_backward(c["dY"], c["dH"], f["H"], f["rstd"], c["gamma"], c["X"], c["gate"], c["post_gamma"], f["post_rstd"], 0.5)
    b = ce.foak_residual_norm_backward(near["dY"], near["dH"], f["H"], f["rstd"], near["gamma"], X=far(c["X"]), post_rstd=f["post_rstd"], **how)
    for k, w in want.items():
        ref.assert_close(b[k], w, k)
    b = ce.foak_residual_norm_backward(near["dY"], near["dH"], f["H"], f["rstd"], near["gamma"], X=near["X"], post_rstd=f["post_rstd"], dR=far(None), **how)
    for k, w in want.items():
        ref.assert_close(b[k], w, k)


def test_rotary_tokens_past_four_gigabytes(cuda_lib):
    ce, T, H, d = cuda_lib, 35007, 240, 256
    plan = ce.foak_rotary_plan(d, base=500000.0)
    few = torch.randn(REPEAT, H, d, device="cuda").to(BF16)
    rows = torch.arange(T, device="cuda") % REPEAT
    q, pos = few[rows], rows * 1000
    assert q.numel() * 2 > 2 ** 32
    out, _ = ce.foak_rotary_apply(plan, pos, q)
    alone, _ = ce.foak_rotary_apply(plan, pos[:REPEAT].contiguous(), few)
    assert torch.equal(out[:REPEAT], alone)
    _same_rows(out, "out")
    ce.foak_rotary_apply(plan, pos, q, q_out=q)
    assert torch.equal(q[-1], out[-1]) and torch.equal(q[:REPEAT], alone)


def test_rotary_calls_of_more_items_than_a_launch_takes(cuda_lib):
    """Heads of odd size, an element at a time: nine tokens are 1.2e9 items, two launches."""
    ce, T, H, d = cuda_lib, 9, 4096, 65535
    plan = ce.foak_rotary_plan(65534, base=10000.0)
    one = torch.randn(1, H, d, device="cuda").to(BF16)
    q = one.expand(T, H, d).contiguous()
    pos = torch.full((T,), 12345, dtype=torch.int64, device="cuda")
    alone, _ = ce.foak_rotary_apply(plan, pos[:1].contiguous(), one)
    ce.foak_rotary_apply(plan, pos, q, q_out=q)
    for t in range(T):
        assert torch.equal(q[t], alone[0]), t
    turns = [t % 2 ** 64 for t in plan.turns.tolist()]
    ref.assert_close(alone[:, :2], ref.rotate(one[:, :2], [12345], turns, 65534, False), "a head")
