"""Refusals of the log-probability and distillation calls, and the float64 references
they are checked against.  No GPU: every call here returns before the first CUDA call."""
import math

import numpy as np
import pytest
import torch

import row_ops_ref as ref

FAKE = 0x10000  # fake device address, never touched


@pytest.fixture(scope="module")
def so():
    import __graft_entry__

    __graft_entry__._build_module().build()
    import cross_entropy_loss_gb300 as ce

    return ce


def _lp(so, logits=FAKE, dtype=1, ld=1000, labels=FAKE, N=4, V=1000, T=1.0, K=5, logp=FAKE, ent=FAKE, lse=FAKE,
        stats=FAKE, top=FAKE, ids=FAKE, err=None, ws=FAKE, wsb=256):
    return so.lib.foak_logprobs_forward(logits, dtype, ld, labels, N, V, -100, T, K, logp, ent, lse, stats, top, ids,
                                        err, ws, wsb, None)


def test_logprobs_forward_refusals(so):
    I, U = so.FOAK_ERR_INVALID_ARG, so.FOAK_ERR_UNSUPPORTED
    assert _lp(so, dtype=2) == U
    assert _lp(so, ld=999) == I and _lp(so, N=-1) == I and _lp(so, V=0) == I
    assert _lp(so, logits=None) == I and _lp(so, logits=FAKE + 1) == I and _lp(so, labels=FAKE + 4) == I
    assert _lp(so, labels=None) == I                      # a log probability of no token
    for T in (0.0, -1.0, math.nan, math.inf, 1e-7, 1e7):
        assert _lp(so, T=T) == I
    assert _lp(so, K=-1) == I and _lp(so, K=1001) == I and _lp(so, K=257) == U
    assert _lp(so, V=262145, ld=262145) == U              # top tokens of a row past their limit
    assert _lp(so, top=None) == I and _lp(so, ids=None) == I
    for k in ("logp", "ent", "lse", "top", "ids", "err"):
        assert _lp(so, **{k: FAKE + 2}) == I
    assert _lp(so, stats=FAKE + 4) == I
    assert _lp(so, ws=None) == so.FOAK_ERR_WORKSPACE and _lp(so, ws=FAKE + 16) == so.FOAK_ERR_WORKSPACE
    assert _lp(so, wsb=255) == so.FOAK_ERR_WORKSPACE
    assert int(so.lib.foak_logprobs_workspace_size()) == 256
    so.lib.foak_test_fail_next_launches(1)
    try:
        assert _lp(so) == so.FOAK_ERR_CUDA
    finally:
        so.lib.foak_test_fail_next_launches(0)


def _lpb(so, dl=FAKE, logits=FAKE, labels=FAKE, N=4, T=1.0, stats=FAKE, gl=FAKE, ent=FAKE, gh=FAKE, err=None):
    return so.lib.foak_logprobs_backward(dl, logits, 1, 1000, labels, N, 1000, -100, T, stats, gl, ent, gh, err, None)


def test_logprobs_backward_refusals(so):
    I = so.FOAK_ERR_INVALID_ARG
    assert _lpb(so, dl=None) == I and _lpb(so, stats=None) == I and _lpb(so, labels=None) == I
    assert _lpb(so, dl=FAKE + 2) == I                     # another offset modulo 16 bytes
    assert _lpb(so, ent=None) == I                        # an entropy gradient without the entropy
    assert _lpb(so, T=0.0) == I and _lpb(so, stats=FAKE + 4) == I and _lpb(so, gl=FAKE + 1) == I
    so.lib.foak_test_fail_next_launches(1)
    try:
        assert _lpb(so) == so.FOAK_ERR_CUDA
    finally:
        so.lib.foak_test_fail_next_launches(0)


def _ds(so, which="fwd_bwd", logits=FAKE, dl=FAKE, dtype=1, ld=1000, labels=FAKE, N=4, V=1000, ids=FAKE, t=FAKE, ldt=8,
        K=8, cew=0.5, kdw=1.0, T=2.0, loss=FAKE, ce=None, kd=None, stats=FAKE, go=None, ws=FAKE, wsb=1 << 16):
    if which == "forward":
        return so.lib.foak_distill_forward(logits, dtype, ld, labels, N, V, -100, ids, t, ldt, K, 1, cew, kdw, T, 0.0,
                                           loss, ce, kd, stats, None, None, ws, wsb, None)
    if which == "fwd_bwd":
        return so.lib.foak_distill_fwd_bwd(logits, dl, dtype, ld, labels, N, V, -100, ids, t, ldt, K, 1, cew, kdw, T,
                                           1.0, 0.0, loss, ce, kd, None, None, ws, wsb, None)
    return so.lib.foak_distill_backward(dl, logits, dtype, ld, labels, N, V, -100, ids, t, ldt, K, 1, cew, kdw, T, stats,
                                        go, 0.0, None, None)


@pytest.mark.parametrize("which", ["forward", "fwd_bwd", "backward"])
def test_distill_refusals(so, which):
    I, U, W = so.FOAK_ERR_INVALID_ARG, so.FOAK_ERR_UNSUPPORTED, so.FOAK_ERR_WORKSPACE
    call = lambda **kw: _ds(so, which, **kw)  # noqa: E731
    assert call(dtype=7) == U and call(ld=10) == I and call(N=-1) == I and call(logits=None) == I
    assert call(ids=None) == I and call(t=None) == I and call(ids=FAKE + 2) == I and call(t=FAKE + 2) == I
    assert call(K=0) == I and call(ldt=7) == I and call(K=257, ldt=300) == U
    assert call(labels=None) == I                         # cross-entropy without labels
    for bad in (math.nan, math.inf):
        assert call(cew=bad) == I and call(kdw=bad) == I and call(T=bad) == I
    if which != "backward":
        assert call(loss=None) == I and call(ce=FAKE + 1) == I and call(kd=FAKE + 2) == I
        assert call(ws=None) == W and call(wsb=256) == W
    if which != "forward":
        assert call(dl=None) == I and call(dl=FAKE + 4) == I
    if which != "fwd_bwd":
        assert call(stats=FAKE + 8) == I
    so.lib.foak_test_fail_next_launches(1)
    try:
        assert call() == so.FOAK_ERR_CUDA
    finally:
        so.lib.foak_test_fail_next_launches(0)


def test_binding_refusals(so):
    x = torch.zeros(3, 10)
    with pytest.raises(ValueError):
        so.foak_logprobs_forward(x, None)                 # not on a CUDA device
    ids, t = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    dev = x.device
    assert so._teacher_args(ids, t, 3, dev) == (2, 2)
    for a, b in ((ids.long(), t), (ids, t.double()), (ids[:2], t), (ids, t[:, :1]), (ids[:, :0], t[:, :0]),
                 (torch.zeros(3, 300, dtype=torch.int32), torch.zeros(3, 300)),
                 (torch.zeros(2, 3, dtype=torch.int32).t(), torch.zeros(2, 3).t()), (ids, torch.zeros(3, 9)[:, :2])):
        with pytest.raises(ValueError):
            so._teacher_args(a, b, 3, dev)
    with pytest.raises(ValueError):
        so._row_vector(torch.zeros(3, dtype=torch.float64), 3, dev, "v")
    with pytest.raises(ValueError):
        so._dlogits_arg(torch.zeros(3, 11), x, 3, 10, 10)


def test_reference_gradients_against_differences():
    """The references' own gradients, by central differences in float64."""
    N, V, K, h = 2, 23, 6, 1e-5
    x = ref.make_logits(N, V, torch.float32, seed=1, sigma=1.0).double()
    r = np.random.default_rng(0)
    y = torch.from_numpy(r.integers(0, V, N))
    ids = torch.from_numpy(np.stack([r.permutation(V)[:K] for _ in range(N)])).int()
    t = torch.from_numpy(r.standard_normal((N, K))).float()
    gl, gh = torch.tensor([1.5, -0.5]), torch.tensor([0.25, 2.0])
    for T in (1.0, 2.0):
        want = ref.logprobs(x, y, 0, T)
        g, _ = ref.logprobs_grad(want, y, T, gl, gh)
        full = ref.distill(x, y, ids, t, T, 0.3, 1.2, True)
        for i in range(N):
            for j in range(V):
                up, dn = x.clone(), x.clone()
                up[i, j] += h
                dn[i, j] -= h
                fu, fd = ref.logprobs(up, y, 0, T), ref.logprobs(dn, y, 0, T)
                num = (gl[i].double() * (fu["logp"] - fd["logp"])[i] + gh[i].double() * (fu["entropy"] - fd["entropy"])[i]) / (2 * h)
                assert abs(float(num - g[i, j])) < 1e-8
                num = (ref.distill(up, y, ids, t, T, 0.3, 1.2, True)["loss"] - ref.distill(dn, y, ids, t, T, 0.3, 1.2, True)["loss"]) / (2 * h)
                assert abs(num - float(full["dlogits"][i, j])) < 1e-8


def test_reference_bounds_notice_a_planted_mistake():
    """A gradient without its entropy term, and a top list with two tokens swapped, are outside the bounds."""
    x = ref.make_logits(4, 500, torch.float32, seed=2)
    y = torch.tensor([1, 2, 3, 4])
    want = ref.logprobs(x, y, 5, 1.0)
    g, size = ref.logprobs_grad(want, y, 1.0, torch.ones(4), torch.ones(4))
    wrong, _ = ref.logprobs_grad(want, y, 1.0, torch.ones(4), None)
    ref.grad_close(g.float(), g, size)
    with pytest.raises(AssertionError):
        ref.grad_close(wrong.float(), g, size)
    swapped = want["top_ids"].clone()
    swapped[0, [0, 1]] = swapped[0, [1, 0]]
    assert not torch.equal(swapped, want["top_ids"])
