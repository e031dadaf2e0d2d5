"""GPU parity of the residual norms, forward and backward, against 64-bit references with derived bounds."""
import pytest
import torch

import block_ops_ref as ref

pytestmark = pytest.mark.gpu

GATES = ("none", "channel", "row", "full")


def _cuda(c):
    return {k: None if v is None else v.cuda() for k, v in c.items()}


def _check_forward(ce, c, scale, eps=1e-5, post_eps=1e-6, gamma=True, **given):
    g = _cuda(c)
    out = ce.foak_residual_norm_forward(g["X"], g["R"], g["gamma"] if gamma else None, gate=g["gate"], post_gamma=g["post_gamma"], scale=scale, eps=eps, post_eps=post_eps, **given)
    want = ref.norm_forward(c["X"], c["R"], c["gamma"] if gamma else None, c["gate"], c["post_gamma"], scale, eps, post_eps)
    for k in ("H", "Y", "rstd", "post_rstd"):
        assert (out[k] is None) == (k not in want), k
        if k in want:
            ref.assert_close(out[k], want[k], k)
    return out


def _saved(c, scale):
    """What a forward leaves, from the reference: H in the rows' type, float32 rstd and post_rstd."""
    f = ref.norm_forward(c["X"], c["R"], c["gamma"], c["gate"], c["post_gamma"], scale, 1e-5, 1e-6)
    return f["H"][0].to(c["X"].dtype), f["rstd"][0].float(), f["post_rstd"][0].float() if "post_rstd" in f else None


def _check_backward(ce, c, scale, with_dY=True, with_dH=True, **given):
    H, rstd, post_rstd = _saved(c, scale)
    dY, dH = (c["dY"] if with_dY else None), (c["dH"] if with_dH else None)
    want = ref.norm_backward(dY, dH, H, rstd, c["gamma"], c["X"], c["gate"], c["post_gamma"], post_rstd, scale)
    g = _cuda(c)
    out = ce.foak_residual_norm_backward(g["dY"] if with_dY else None, g["dH"] if with_dH else None, H.cuda(), rstd.cuda(), g["gamma"], X=g["X"], gate=g["gate"], post_gamma=g["post_gamma"], post_rstd=None if post_rstd is None else post_rstd.cuda(), scale=scale, **given)
    for k in ("dR", "dX", "dgamma", "dgate", "dpost_gamma"):
        assert (out[k] is None) == (k not in want), k
        if k in want:
            ref.assert_close(out[k], want[k], k)
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("N,D", [(1, 8), (3, 40), (37, 520), (5, 4096), (2, 8200), (1, 32768), (700, 64)])
def test_forward(cuda_lib, N, D, gate, post, dtype):
    _check_forward(cuda_lib, ref.make_norm(N, D, dtype, gate, post, seed=N + D), 0.22)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("N,D", [(1, 8), (3, 40), (37, 520), (5, 4096), (2, 8200), (1, 32768), (700, 64)])
def test_backward(cuda_lib, N, D, gate, post, dtype):
    _check_backward(cuda_lib, ref.make_norm(N, D, dtype, gate, post, seed=N + D), 0.22)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1000, 2048, 4096, 5120, 8192, 16384])
def test_many_rows(cuda_lib, D, dtype):
    """More rows than the GPU has CTAs: every CTA goes round its loop."""
    N = 2500 if D < 8192 else 700
    for gate, post in (("none", False), ("channel", True), ("full", True), ("row", False)):
        c = ref.make_norm(N, D, dtype, gate, post, seed=D)
        _check_forward(cuda_lib, c, 1.0)
        _check_backward(cuda_lib, c, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 4096, 16384])
def test_parts_that_are_left_out(cuda_lib, D, dtype):
    """No norm before the next block, no gradient along the stream, gradients that nobody wants."""
    ce = cuda_lib
    for gate, post in (("none", False), ("channel", True), ("row", True), ("full", False), ("row", False)):
        c = ref.make_norm(19, D, dtype, gate, post, seed=3)
        _check_forward(ce, c, 0.5, gamma=False)
        _check_backward(ce, c, 0.5, with_dH=False)
        _check_backward(ce, c, 0.5, with_dY=False)
        H, rstd, post_rstd = _saved(c, 0.5)
        g = _cuda(c)
        part = ce.foak_residual_norm_backward(g["dY"], g["dH"], H.cuda(), rstd.cuda(), g["gamma"], X=g["X"], gate=g["gate"], post_gamma=g["post_gamma"], post_rstd=None if post_rstd is None else post_rstd.cuda(), scale=0.5, want_dX=False, want_dgate=False, want_dgamma=False)
        # another variant, with its sums in another order: within the same bound
        ref.assert_close(part["dR"], ref.norm_backward(c["dY"], c["dH"], H, rstd, c["gamma"], c["X"], c["gate"], c["post_gamma"], post_rstd, 0.5)["dR"], "dR")
        assert part["dX"] is None and part["dgate"] is None and part["dgamma"] is None and part["dpost_gamma"] is None


def test_plain_residual_shares_its_gradient(cuda_lib):
    c = ref.make_norm(9, 256, "bf16", "none", False, seed=1)
    out = _check_backward(cuda_lib, c, 1.0)
    assert out["dX"] is out["dR"]
    own = _check_backward(cuda_lib, c, 1.0, dX=torch.empty(9, 256, dtype=torch.bfloat16, device="cuda"))
    assert own["dX"] is not own["dR"] and torch.equal(own["dX"], own["dR"])


@pytest.mark.parametrize("D", [512, 4096, 16384])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_row_strides(cuda_lib, D, dtype):
    """Rows inside wider ones, each tensor with a stride of its own; nothing is written between them."""
    ce, N, dt = cuda_lib, 21, ref.DT[dtype]
    c = ref.make_norm(N, D, dtype, "full", True, seed=5)
    wide = {}

    def room(name, pad, fill=7.0):
        wide[name] = torch.full((N, D + pad), fill, dtype=dt, device="cuda")
        return wide[name][:, 8 : 8 + D]

    def put(name, pad):
        room(name, pad).copy_(c[name])
        return wide[name][:, 8 : 8 + D]

    X, R, gate, dY, dH = (put(n, 16 + 8 * i) for i, n in enumerate(("X", "R", "gate", "dY", "dH")))
    H, Y, dR, dX = (room(n, 56 + 8 * i) for i, n in enumerate(("H", "Y", "dR", "dX")))
    gamma, pg = c["gamma"].cuda(), c["post_gamma"].cuda()
    out = ce.foak_residual_norm_forward(X, R, gamma, gate=gate, post_gamma=pg, scale=0.7, eps=1e-5, post_eps=1e-6, H=H, Y=Y)
    want = ref.norm_forward(c["X"], c["R"], c["gamma"], c["gate"], c["post_gamma"], 0.7, 1e-5, 1e-6)
    for k in ("H", "Y", "rstd", "post_rstd"):
        ref.assert_close(out[k], want[k], k)
    back = ce.foak_residual_norm_backward(dY, dH, H, out["rstd"], gamma, X=X, gate=gate, post_gamma=pg, post_rstd=out["post_rstd"], scale=0.7, dR=dR, dX=dX)
    want = ref.norm_backward(c["dY"], c["dH"], H, out["rstd"], c["gamma"], c["X"], c["gate"], c["post_gamma"], out["post_rstd"], 0.7)
    for k, w in want.items():
        ref.assert_close(back[k], w, k)
    for name in ("H", "Y", "dR", "dX"):
        assert bool((wide[name][:, :8] == 7.0).all()) and bool((wide[name][:, 8 + D :] == 7.0).all()), name


@pytest.mark.parametrize("D", [512, 4096, 16384])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(cuda_lib, D, dtype):
    ce, N = cuda_lib, 400
    for gate, post in (("none", False), ("full", True)):
        c = ref.make_norm(N, D, dtype, gate, post, seed=8)
        how = dict(gate=c["gate"] if c["gate"] is None else c["gate"].cuda(), post_gamma=c["post_gamma"] if not post else c["post_gamma"].cuda(), scale=0.3)
        gamma = c["gamma"].cuda()
        plain = ce.foak_residual_norm_forward(c["X"].cuda(), c["R"].cuda(), gamma, **how)
        for h_is, y_is in (("R", "X"), ("X", "R"), ("R", None), ("X", None)):
            t = {"X": c["X"].cuda(), "R": c["R"].cuda()}
            out = ce.foak_residual_norm_forward(t["X"], t["R"], gamma, H=t[h_is], Y=t.get(y_is), **how)
            assert out["H"] is t[h_is] and torch.equal(out["H"], plain["H"]) and torch.equal(out["Y"], plain["Y"]), (h_is, y_is)
        rs, pr = plain["rstd"], plain["post_rstd"]
        args = dict(X=c["X"].cuda(), post_rstd=pr, **how)
        a = ce.foak_residual_norm_backward(c["dY"].cuda(), c["dH"].cuda(), plain["H"], rs, gamma, **args)
        for r_is, x_is in (("dH", "dY"), ("dY", "dH"), ("dH", "X"), ("dY", "H")):
            t = {"dY": c["dY"].cuda(), "dH": c["dH"].cuda(), "X": c["X"].cuda(), "H": plain["H"].clone()}
            b = ce.foak_residual_norm_backward(t["dY"], t["dH"], t["H"], rs, gamma, dR=t[r_is], dX=t[x_is], **{**args, "X": t["X"]})
            for k in a:
                assert (a[k] is None and b[k] is None) or torch.equal(a[k], b[k]), (k, r_is, x_is)


def test_values_at_the_edges(cuda_lib):
    """Rows that cancel, rows of zeros, infinities and NaN that stay in their rows."""
    ce = cuda_lib
    for dtype in ("bf16", "f32"):
        c = ref.make_norm(6, 4096, dtype, "none", False, seed=11, cancel=True)
        _check_forward(ce, c, 1.0)
        c = ref.make_norm(6, 1024, dtype, "full", True, seed=12)
        c["X"][1] = 0
        c["R"][1] = 0
        c["X"][2, 5] = float("inf")
        c["R"][3, 7] = float("nan")
        c["gate"][4, 1] = float("-inf")
        c["R"][5] = 0
        c["gate"][5] = 0
        g = _cuda(c)
        out = ce.foak_residual_norm_forward(g["X"], g["R"], g["gamma"], gate=g["gate"], post_gamma=g["post_gamma"], scale=1.0, eps=1e-5)
        want = ref.norm_forward(c["X"], c["R"], c["gamma"], c["gate"], c["post_gamma"], 1.0, 1e-5, 1e-5)
        for k in ("H", "Y", "rstd", "post_rstd"):
            got, w = out[k].cpu().double(), want[k][0]
            assert torch.equal(got.isnan(), w.isnan()) and torch.equal(got.isinf(), w.isinf()), k
            for i in (0, 1, 5):
                ref.assert_close(out[k][i : i + 1], (want[k][0][i : i + 1], want[k][1][i : i + 1]), k)


def test_empty_batch(cuda_lib):
    ce = cuda_lib
    for gate in ("none", "channel", "full", "row"):
        c = _cuda(ref.make_norm(0, 64, "bf16", gate, True, seed=1))
        out = ce.foak_residual_norm_forward(c["X"], c["R"], c["gamma"], gate=c["gate"], post_gamma=c["post_gamma"])
        assert out["H"].shape == out["Y"].shape == (0, 64)
        back = ce.foak_residual_norm_backward(c["dY"], c["dH"], out["H"], out["rstd"], c["gamma"], X=c["X"], gate=c["gate"], post_gamma=c["post_gamma"], post_rstd=out["post_rstd"])
        assert back["dR"].shape == (0, 64) and not back["dgamma"].any() and not back["dpost_gamma"].any()
        if gate == "channel":
            assert not back["dgate"].any()


def test_gradients_against_differences(cuda_lib):
    """Central differences of the 64-bit forward, step 1e-5: their error is about 1e-9."""
    ce, N, D = cuda_lib, 3, 16
    for gate, post in (("none", False), ("channel", True), ("row", True), ("full", True), ("channel", False), ("row", False)):
        c = ref.make_norm(N, D, "f32", gate, post, seed=21)
        names = [k for k in ("R", "X", "gamma", "gate", "post_gamma") if c[k] is not None]
        d = {k: c[k].double() for k in names}

        def loss(t):
            f = ref.norm_forward(t["X"], t["R"], t["gamma"], t.get("gate"), t.get("post_gamma"), 0.6, 1e-5, 1e-6)
            return float((f["Y"][0] * c["dY"].double()).sum() + (f["H"][0] * c["dH"].double()).sum())

        out = _check_backward(ce, c, 0.6)
        for k in names:
            got = out["d" + k].cpu().double().reshape(d[k].shape)
            for j in range(d[k].numel()):
                lo, hi = d[k].clone(), d[k].clone()
                lo.view(-1)[j] -= 1e-5
                hi.view(-1)[j] += 1e-5
                slope = (loss({**d, k: hi}) - loss({**d, k: lo})) / 2e-5
                # sums of at most 48 products of float32 values of order one to ten
                assert abs(float(got.reshape(-1)[j]) - slope) <= 1e-8 + 100 * ref.U * (abs(slope) + 10.0), (gate, post, k, j)


def test_run_to_run(cuda_lib):
    ce = cuda_lib
    c = _cuda(ref.make_norm(1500, 2048, "bf16", "channel", True, seed=2))
    f = ce.foak_residual_norm_forward(c["X"], c["R"], c["gamma"], gate=c["gate"], post_gamma=c["post_gamma"])
    outs = [ce.foak_residual_norm_backward(c["dY"], c["dH"], f["H"], f["rstd"], c["gamma"], X=c["X"], gate=c["gate"], post_gamma=c["post_gamma"], post_rstd=f["post_rstd"]) for _ in range(3)]
    for o in outs[1:]:
        assert all(torch.equal(o[k], outs[0][k]) for k in o)


def test_refusals_of_the_binding(cuda_lib):
    ce = cuda_lib
    X, g = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    rs = torch.ones(4, device="cuda")
    bad = [
        lambda: ce.foak_residual_norm_forward(X, X[:2], g),
        lambda: ce.foak_residual_norm_forward(X, X.bfloat16(), g),
        lambda: ce.foak_residual_norm_forward(X, X.cpu(), g),
        lambda: ce.foak_residual_norm_forward(X, X, g[:32]),
        lambda: ce.foak_residual_norm_forward(X, X, g, gate=torch.ones(1, 64, device="cuda")),
        lambda: ce.foak_residual_norm_forward(X, X, None, Y=X.clone()),
        lambda: ce.foak_residual_norm_forward(X.t(), X.t(), None),
        lambda: ce.foak_residual_norm_backward(None, None),
        lambda: ce.foak_residual_norm_backward(X, None),
        lambda: ce.foak_residual_norm_backward(X, None, X, rs[:2], g),
        lambda: ce.foak_residual_norm_backward(X, None, X, rs, g, gate=g),
        lambda: ce.foak_residual_norm_backward(X, None, X, rs, g, X=X, post_gamma=g),
        lambda: ce.foak_residual_norm_backward(X, None, X, rs, g, workspace_tensor=torch.zeros(1 << 22, dtype=torch.uint8)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    for call in (lambda: ce.foak_residual_norm_forward(X[:, :60], X[:, :60], g[:60]),  # D % 8
                 lambda: ce.foak_residual_norm_forward(X, X, g, H=X, Y=X),
                 lambda: ce.foak_residual_norm_forward(X, X, g, scale=float("nan")),
                 lambda: ce.foak_residual_norm_forward(X, X, g, eps=-1.0),
                 lambda: ce.foak_residual_norm_backward(X, None, X, rs, g, scale=2.0, dR=X, dX=X),
                 lambda: ce.foak_residual_norm_backward(X, None, X, rs, g, workspace_tensor=torch.zeros(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ce.FoakError):
            call()
