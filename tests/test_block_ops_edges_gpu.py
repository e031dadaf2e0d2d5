"""Residual norms and rotary positions where the other tests do not go: angles near zero, the backward's kernels for
any rows, gates without a gradient, rows over a cluster, sums over very many rows."""
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


# ------------------------------------------------------------------- residual norms
# The references' bounds go by chains of 80 additions within a row and N / 128 + 60 over the rows (block_ops_ref).
# Within a row the two kernels for any rows add D / 256 elements a thread and 10 more: 80 is enough up to D = 16384.
# Over the rows the one-pass kernel has a group for each of the clusters that are resident, 2432 of them at most: N /
# groups additions, then 76 + 32 by the 32 warps that join them.  A cluster of C CTAs fits every 2 C SMs at least once (a part
# of the GPU of n >= C SMs that share clusters has n / C of them, rounded down, which is more than n / 2 C).
def _sum_chain(N, D, dtype):
    vectors = D * (2 if dtype == "bf16" else 4) // 16
    cluster = next(c for c in (1, 2, 4, 8) if -(-vectors // c) <= 1024)
    groups = min(N, torch.cuda.get_device_properties(0).multi_processor_count // (2 * cluster))
    return -(-N // groups) + 76 + 32 + 8


def _case(N, D, dtype, gate, post, seed, scale):
    """Operands on the CPU and what a forward leaves of them."""
    c = ref.make_norm(N, D, dtype, gate, post, seed)
    f = ref.norm_forward(c["X"], c["R"], c["gamma"], c["gate"], c["post_gamma"], scale, 1e-5, 1e-6)
    c.update(H=f["H"][0].to(ref.DT[dtype]), rstd=f["rstd"][0].float(), post_rstd=f["post_rstd"][0].float() if post else None)
    return c


def _want(c, scale, dtype, with_dY=True, with_dH=True):
    """The reference's gradients; the bounds of the sums over the rows by the kernel's own chain of additions."""
    dY, dH = (c["dY"] if with_dY else None), (c["dH"] if with_dH else None)
    want = ref.norm_backward(dY, dH, c["H"], c["rstd"], c["gamma"], c["X"], c["gate"], c["post_gamma"], c["post_rstd"], scale)
    N, D = c["X"].shape
    more = max(0.0, _sum_chain(N, D, dtype) / (ref.row_chain(N) + 8) - 1.0)
    for k in ("dgamma", "dgate", "dpost_gamma"):
        if k in want and want[k][0].dim() == 1:
            want[k] = (want[k][0], want[k][1] * (1.0 + more))
    return want


def _backward(ce, c, scale, with_dY=True, with_dH=True, place=lambda name, t: t, **how):
    g = {k: None if v is None else place(k, v.cuda()) for k, v in c.items()}
    return ce.foak_residual_norm_backward(g["dY"] if with_dY else None, g["dH"] if with_dH else None, g["H"], g["rstd"], g["gamma"], X=g["X"], gate=g["gate"], post_gamma=g["post_gamma"], post_rstd=g["post_rstd"], scale=scale, **how)


def _compare(out, want, names):
    for k in ("dR", "dX", "dgamma", "dgate", "dpost_gamma"):
        assert (out[k] is None) == (k not in names), k
        if k in names:
            ref.assert_close(out[k], want[k], k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,D", [(1, 64), (37, 520), (2500, 2048), (5000, 264), (400, 8200), (300, 16384)])
def test_gradients_under_a_gate_without_the_gates_own(cuda_lib, N, D, dtype):
    """A gate that is not trained: every other gradient as with it, from one row to many a CTA."""
    for gate, post in (("channel", False), ("row", False), ("full", False), ("channel", True), ("row", True), ("full", True)):
        c = _case(N, D, dtype, gate, post, 7, 0.6)
        for with_dY, with_dH in ((True, True), (True, False), (False, True)):
            names = {"dR", "dX"} | ({"dgamma"} if with_dY else set()) | ({"dpost_gamma"} if post else set())
            want = _want(c, 0.6, dtype, with_dY, with_dH)
            _compare(_backward(cuda_lib, c, 0.6, with_dY, with_dH, want_dgate=False), want, names)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["none", "channel", "row", "full"])
def test_gradients_of_far_rows(cuda_lib, gate, dtype):
    """Four rows, one operand's 4 GiB apart, with and without the norm after the block: all gradients."""
    N, D, dt = 4, 1032, ref.DT[dtype]
    ld = 2 ** 32 // dt.itemsize + 8
    room = torch.empty((N - 1) * ld + D, dtype=dt, device="cuda").as_strided((N, D), (ld, 1))
    for post in (False, True):
        c = _case(N, D, dtype, gate, post, 9, 0.7)
        want = _want(c, 0.7, dtype)
        far = {"dH": lambda name, t: room.copy_(t) if name == "dH" else t}
        if gate == "full":
            far["gate"] = lambda name, t: room.copy_(t) if name == "gate" else t
        for place in far.values():
            _compare(_backward(cuda_lib, c, 0.7, place=place), want, set(want))
        b = _backward(cuda_lib, c, 0.7, dX=room)
        assert b["dX"] is room
        _compare(b, want, set(want))


def _any_rows(ce, c, scale, without):
    """The C call with one operand left out whose stride is past 32 bits: the kernels for any rows, however many."""
    N, D = c["X"].shape
    g = {k: v.cuda() for k, v in c.items() if v is not None and k != without}
    like, kind = g["X"], {(): 0, (D,): 1, (N, 1): 2, (N, D): 3}[tuple(c["gate"].shape) if c["gate"] is not None else ()]
    out = dict(dR=torch.empty_like(like), dX=torch.empty_like(like))
    if without != "dY":
        out["dgamma"] = torch.empty(D, device="cuda")
    if kind:
        out["dgate"] = torch.empty_like(like) if kind == 3 else torch.empty(D if kind == 1 else N, device="cuda")
    if c["post_gamma"] is not None:
        out["dpost_gamma"] = torch.empty(D, device="cuda")
    ws = torch.empty(ce.foak_residual_norm_workspace_size(N, D), dtype=torch.uint8, device="cuda")
    at = {k: v.data_ptr() for k, v in (g | out).items()}.get
    ld = lambda name: 2 ** 40 if name == without else D  # noqa: E731
    st = ce.lib.foak_residual_norm_backward(
        at("dY"), ld("dY"), at("dH"), ld("dH"), at("H"), D, at("X"), D, ce._DT[like.dtype], N, D, at("gate"), kind, 1 if kind == 2 else D, at("post_gamma"), at("gamma"),
        at("post_rstd"), at("rstd"), scale, at("dR"), D, at("dX"), D, at("dgamma"), at("dgate"), D, at("dpost_gamma"), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == ce.FOAK_OK
    return {**dict.fromkeys(("dgamma", "dgate", "dpost_gamma")), **out}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate,post", [("none", False), ("channel", False), ("row", False), ("full", False), ("none", True), ("channel", True), ("row", True), ("full", True)])
def test_gradients_by_the_kernels_for_any_rows(cuda_lib, gate, post, dtype):
    """A row, a few, and several for each of their CTAs; rows of one thread's vector and of many."""
    for N, D in ((1, 8), (200, 16384), (5000, 264)):
        c = _case(N, D, dtype, gate, post, 11, 0.4)
        for without in ("dH", "dY"):
            want = _want(c, 0.4, dtype, with_dY=without != "dY", with_dH=without != "dH")
            out = _any_rows(cuda_lib, c, 0.4, without)
            _compare(out, want, set(want))


@pytest.mark.parametrize("D,dtype", [(20480, "f32"), (32768, "f32"), (17408, "bf16"), (32768, "bf16")])
def test_rows_over_a_cluster(cuda_lib, D, dtype):
    """Rows over eight CTAs, and over four, many of them for each cluster."""
    N = 170
    for gate, post in (("none", False), ("channel", True), ("row", False), ("full", True)):
        c = _case(N, D, dtype, gate, post, 13, 0.8)
        want = _want(c, 0.8, dtype)
        out = _backward(cuda_lib, c, 0.8)
        _compare(out, want, set(want))
        again = _backward(cuda_lib, c, 0.8)
        assert all(torch.equal(out[k], again[k]) for k in want)


@pytest.mark.parametrize("N,D,dtype", [(20011, 32768, "f32"), (60013, 16384, "bf16"), (500009, 64, "f32")])
def test_sums_over_many_rows(cuda_lib, N, D, dtype):
    """The gradients that are summed over the rows, of seven rows over and over, against the seven's own by how often
    each is there."""
    seven = _case(7, D, dtype, "channel", True, 15, 0.3)
    rows = torch.arange(N, device="cuda") % 7
    g = {k: v.cuda() for k, v in seven.items()}
    for k in ("X", "dY", "dH", "H", "rstd", "post_rstd"):
        g[k] = g[k][rows]
    out = cuda_lib.foak_residual_norm_backward(g["dY"], g["dH"], g["H"], g["rstd"], g["gamma"], X=g["X"], gate=g["gate"], post_gamma=g["post_gamma"], post_rstd=g["post_rstd"], scale=0.3, dR=g["dH"], dX=g["dY"])
    sums = {}
    for i in range(7):
        one = {k: v[i : i + 1] if k in ("X", "dY", "dH", "H", "rstd", "post_rstd") else v for k, v in seven.items()}
        want = ref.norm_backward(one["dY"], one["dH"], one["H"], one["rstd"], one["gamma"], one["X"], one["gate"], one["post_gamma"], one["post_rstd"], 0.3)
        times = (N - 1 - i) // 7 + 1
        for k in ("dgamma", "dgate", "dpost_gamma"):
            value, bound = want[k]
            size = times * (bound + _sum_chain(N, D, dtype) * ref.U * value.abs())
            before = sums.get(k, (0.0, 0.0))
            sums[k] = (before[0] + times * value, before[1] + size)
    for k, want in sums.items():
        ref.assert_close(out[k], want, k)
