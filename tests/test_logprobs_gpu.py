"""The log-probability calls against float64: values, entropies, top tokens and gradients
over types, row shapes, clusters, masks and ties; bounds derived in row_ops_ref."""
import math

import numpy as np
import pytest
import torch

import row_ops_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _labels(N, V, seed, n_ignore=0):
    r = np.random.default_rng(seed + 1000)
    y = torch.from_numpy(r.integers(0, V, N))
    if n_ignore:
        y[torch.from_numpy(r.permutation(N)[:n_ignore])] = -100
    return y


def _check_forward(ce, x, y, K, T=1.0):
    xd = ref.to_gpu(x)
    out = ce.foak_logprobs_forward(xd, None if y is None else y.cuda(), top_k=K, temperature=T)
    torch.cuda.synchronize()
    want = ref.logprobs(x, y, K, T)
    V = x.shape[1]
    ref.close(out["lse"], want["lse"], ref.value_tol(want["lse"]), "lse")
    ref.close(out["entropy"], want["entropy"], ref.entropy_tol(V), "entropy")
    if y is None:
        assert out["logp"] is None
    else:
        ref.close(out["logp"], want["logp"], ref.value_tol(want["logp"]), "logp")
    if K:
        assert out["top_ids"].dtype == torch.int32
        got = out["top_ids"].cpu().long()
        assert torch.equal(got, want["top_ids"]), (got[(got != want["top_ids"]).any(1)][:2], want["top_ids"][(got != want["top_ids"]).any(1)][:2])
        ref.close(out["top_logprobs"], want["top_logprobs"], ref.value_tol(want["top_logprobs"]), "top_logprobs")
    else:
        assert out["top_ids"] is None and out["top_logprobs"] is None
    assert int(out["err"].item()) == 0
    return xd, out, want


def _check_backward(ce, x, xd, y, out, want, T, seed=0, entropy=True, in_place=False):
    r = np.random.default_rng(seed + 5)
    N = x.shape[0]
    gl = torch.from_numpy(r.standard_normal(N).astype(np.float32))
    gh = torch.from_numpy(r.standard_normal(N).astype(np.float32)) if entropy else None
    dx, err = ce.foak_logprobs_backward(xd, y.cuda(), out["stats"], gl.cuda(), out["entropy"] if entropy else None,
                                        gh.cuda() if entropy else None, temperature=T,
                                        dlogits=xd if in_place else None)
    torch.cuda.synchronize()
    g, size = ref.logprobs_grad(want, y, T, gl, gh)
    ref.grad_close(dx, g, size)
    assert int(err.item()) == 0
    ign = ~want["ok"]
    if ign.any():
        z = dx[ign.cuda()]
        assert not bool(z.float().abs().sum() > 0) and not bool(torch.signbit(z.float()).any())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,V,K", [(1, 1, 1), (3, 2, 2), (5, 7, 3), (4, 31, 31), (2, 33, 20), (9, 1000, 64),
                                   (6, 8192, 20), (5, 32000, 5), (3, 50257, 128), (2, 128256, 20), (1, 128256, 256),
                                   (40, 32000, 20), (90, 50257, 7), (400, 9001, 50), (1000, 2055, 8),
                                   (2, 128256, 100), (64, 128263, 20), (130, 128256, 200), (20, 64131, 3),
                                   (20, 32000, 256), (200, 40001, 161)])
def test_shapes(cuda_lib, dtype, N, V, K):
    x = ref.make_logits(N, V, dtype, seed=N + V)
    y = _labels(N, V, N + V, n_ignore=N // 7)
    T = 0.7 if V % 2 else 1.0
    xd, out, want = _check_forward(cuda_lib, x, y, K, T)
    _check_backward(cuda_lib, x, xd, y, out, want, T, entropy=N % 2 == 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("ld_more,offset", [(0, 1), (1, 0), (3, 5), (8, 0), (13, 7)])
@pytest.mark.parametrize("N,V", [(7, 5003), (300, 1031), (2, 100001), (2, 128263)])
def test_strides_and_offsets(cuda_lib, dtype, ld_more, offset, N, V):
    x = ref.make_logits(N, V, dtype, seed=V + offset, ld=V + ld_more, offset=offset)
    y = _labels(N, V, V, n_ignore=1)
    xd, out, want = _check_forward(cuda_lib, x, y, 17, 1.5)
    _check_backward(cuda_lib, x, xd, y, out, want, 1.5, in_place=offset % 2 == 1)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,V", [(12, 32003), (200, 32003), (1, 128256), (12, 128259), (64, 128256)])
def test_masks(cuda_lib, dtype, N, V):
    """Rows with -inf, the lowest value, one token left, nothing left; mixtures of both masks."""
    low = torch.finfo(dtype).min
    x = ref.make_logits(N, V, dtype, seed=V)
    y = _labels(N, V, V)
    r = np.random.default_rng(3)
    for i in range(N):
        kind = i % 10 if N > 1 else 4
        drop = torch.from_numpy(r.random(V) < 0.5)
        if kind == 0:
            x[i, drop] = -math.inf
        elif kind == 1:
            x[i, drop] = low
        elif kind == 2:
            x[i] = -math.inf
        elif kind == 3:
            x[i] = low
        elif kind == 4:
            keep = x[i, [3, V // 2, V - 1]].clone()
            x[i] = -math.inf
            x[i, [3, V // 2, V - 1]] = keep
        elif kind == 5:
            x[i] = -math.inf
            x[i, drop] = low
        elif kind == 6:
            x[i] = low
            x[i, 5] = -math.inf
            x[i, V - 2] = 1.0
        elif kind == 7:
            x[i] = -math.inf
            x[i, y[i]] = -7.5
    xd, out, want = _check_forward(cuda_lib, x, y, 20)
    if N > 2:
        assert float(out["lse"][2]) == -math.inf and float(out["entropy"][2]) == 0.0
        assert out["top_ids"][2].tolist() == list(range(20))
        np.testing.assert_allclose(float(out["logp"][3]), -math.log(V), atol=ref.EPS + 1e-6)
    _check_backward(cuda_lib, x, xd, y, out, want, 1.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,V,K", [(3, 32000, 20), (200, 32001, 128), (1, 128256, 50), (2, 700, 256), (160, 12000, 256),
                                   (3, 128256, 200), (100, 128256, 20)])
def test_ties_go_to_the_lowest_id(cuda_lib, dtype, N, V, K):
    r = np.random.default_rng(V)
    x = torch.empty(N, V, dtype=dtype)
    for i in range(N):
        kind = i % 5
        if kind == 0:
            x[i] = 3.0  # one value
        elif kind == 1:
            x[i] = torch.from_numpy(r.integers(0, 4, V).astype(np.float32))  # four values
        elif kind == 2:
            x[i] = torch.from_numpy(r.choice([-0.0, 0.0], V).astype(np.float32))  # the two zeros are equal
        elif kind == 3:
            x[i] = torch.arange(V, 0, -1).float().div(64).floor()  # descending, in steps
        else:
            x[i] = torch.arange(V).float().div(V)  # ascending: the largest at the end
    _check_forward(cuda_lib, x, None, K)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [20011, 100003])
def test_magnitudes(cuda_lib, dtype, V):
    """Very large, very small and very spread logits; an outlier far above the rest."""
    x = torch.empty(6, V, dtype=dtype)
    base = ref.make_logits(6, V, F32, seed=5)
    x[0] = base[0] * 1e-30
    x[1] = base[1] * 1e4
    x[2] = base[2] - 3e4
    x[3] = base[3] * 1e30
    x[4] = base[4]
    x[4, 777] = 1e6
    x[5] = base[5] + 2e20
    y = _labels(6, V, 1)
    xd, out, want = _check_forward(cuda_lib, x, y, 33)
    _check_backward(cuda_lib, x, xd, y, out, want, 1.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,V", [(4, 33000), (300, 33000), (4, 128256)])
def test_nan_and_infinity_stay_in_their_row(cuda_lib, dtype, N, V):
    x = ref.make_logits(N, V, dtype, seed=2)
    y = _labels(N, V, 2)
    x[1, 20000] = math.nan
    x[2, 31] = math.inf
    xd = ref.to_gpu(x)
    out = cuda_lib.foak_logprobs_forward(xd, y.cuda(), top_k=5)
    want = ref.logprobs(x, y, 5, 1.0)
    for k in ("logp", "entropy", "lse"):
        v = out[k].cpu()
        assert torch.isnan(v[1:3]).all() and torch.isfinite(v[0]) and torch.isfinite(v[3:]).all()
    assert out["top_ids"][1:3].tolist() == [[-1] * 5] * 2 and torch.isnan(out["top_logprobs"][1:3]).all()
    keep = [0] + list(range(3, N))
    assert torch.equal(out["top_ids"].cpu()[keep].long(), want["top_ids"][keep])
    dx, _ = cuda_lib.foak_logprobs_backward(xd, y.cuda(), out["stats"], torch.ones(N, device="cuda"))
    dx = dx.float().cpu()
    assert torch.isnan(dx[1:3]).all() and torch.isfinite(dx[keep]).all()


def test_long_rows(cuda_lib):
    """Rows past the top tokens' 262144: sums over two million elements; and rows at the limit."""
    x = ref.make_logits(2, 2_000_003, BF16, seed=9)
    y = _labels(2, 2_000_003, 9)
    xd, out, want = _check_forward(cuda_lib, x, y, 0)
    _check_backward(cuda_lib, x, xd, y, out, want, 1.0)
    for dtype in (BF16, F32):
        for N in (1, 160):
            x = ref.make_logits(1, 262144, dtype, seed=N).expand(N, -1).contiguous()
            _check_forward(cuda_lib, x, None, 100)


def test_offsets_past_32_bits(cuda_lib):
    """A row that starts more than 2^32 bytes into the tensor."""
    V, N = 40_009, 60_001
    x = torch.zeros(N, V, dtype=BF16, device="cuda")
    row = ref.make_logits(1, V, BF16, seed=4)
    x[N - 1] = row[0].cuda()
    y = torch.full((N,), -100, dtype=torch.int64, device="cuda")
    y[N - 1] = 12345
    out = cuda_lib.foak_logprobs_forward(x, y, top_k=9)
    want = ref.logprobs(row, torch.tensor([12345]), 9, 1.0)
    assert torch.equal(out["top_ids"][N - 1].cpu().long(), want["top_ids"][0])
    ref.close(out["logp"][N - 1:], want["logp"], ref.value_tol(want["logp"]), "logp")
    assert int((out["top_ids"][: N - 1] != -1).sum()) == 0
    dx, _ = cuda_lib.foak_logprobs_backward(x, y, out["stats"], torch.ones(N, device="cuda"), dlogits=x)
    g, size = ref.logprobs_grad(want, torch.tensor([12345]), 1.0, torch.ones(1), None)
    ref.grad_close(dx[N - 1:], g, size)
    assert int(dx[: N - 1].count_nonzero()) == 0


def test_bad_label_is_reported_and_ignored(cuda_lib):
    x = ref.make_logits(30, 500, F32, seed=1)
    y = _labels(30, 500, 1)
    y[3], y[17] = 500, -1
    xd = ref.to_gpu(x)
    out = cuda_lib.foak_logprobs_forward(xd, y.cuda(), top_k=4)
    want = ref.logprobs(x, y, 4, 1.0)
    assert int(out["err"].item()) == cuda_lib.FOAK_ERRBIT_LABEL_RANGE
    assert torch.equal(out["top_ids"].cpu().long(), want["top_ids"])
    dx, err = cuda_lib.foak_logprobs_backward(xd, y.cuda(), out["stats"], torch.ones(30, device="cuda"))
    assert int(err.item()) == cuda_lib.FOAK_ERRBIT_LABEL_RANGE
    assert int(dx[[3, 17]].count_nonzero()) == 0
    # the next call's word is clean again
    y[3], y[17] = 5, 6
    assert int(cuda_lib.foak_logprobs_forward(xd, y.cuda())["err"].item()) == 0


def test_empty_batch(cuda_lib):
    x = torch.empty(0, 100, dtype=BF16, device="cuda")
    y = torch.empty(0, dtype=torch.int64, device="cuda")
    out = cuda_lib.foak_logprobs_forward(x, y, top_k=3)
    assert out["top_ids"].shape == (0, 3) and int(out["err"].item()) == 0
    dx, err = cuda_lib.foak_logprobs_backward(x, y, out["stats"], out["logp"])
    assert dx.shape == (0, 100) and int(err.item()) == 0


@pytest.mark.parametrize("N", [2, 500])
def test_same_bits_again_and_on_another_stream(cuda_lib, N):
    x = ref.to_gpu(ref.make_logits(N, 32007, BF16, seed=8))
    y = _labels(N, 32007, 8).cuda()
    a = cuda_lib.foak_logprobs_forward(x, y, top_k=40)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.zeros(cuda_lib.foak_ce_workspace_size(0), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    b = cuda_lib.foak_logprobs_forward(x, y, top_k=40, stream=side, workspace_tensor=ws)
    with torch.cuda.stream(side):
        c = cuda_lib.foak_logprobs_forward(x, y, top_k=40, workspace_tensor=ws)
    torch.cuda.synchronize()
    for k in ("logp", "entropy", "lse", "stats", "top_logprobs", "top_ids"):
        assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k]), k


def test_graph_replay(cuda_lib):
    """Forward and backward captured into a graph, replayed on new logits."""
    N, V = 64, 32000
    x = ref.make_logits(N, V, BF16, seed=21)
    xd = ref.to_gpu(x)
    y = _labels(N, V, 21)
    yd = y.cuda()
    gl = torch.ones(N, device="cuda")
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    dx = torch.empty_like(xd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cuda_lib.foak_logprobs_forward(xd, yd, top_k=6, workspace_tensor=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = cuda_lib.foak_logprobs_forward(xd, yd, top_k=6, workspace_tensor=ws)
        cuda_lib.foak_logprobs_backward(xd, yd, out["stats"], gl, dlogits=dx)
    x2 = ref.make_logits(N, V, BF16, seed=22)
    xd.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    want = ref.logprobs(x2, y, 6, 1.0)
    assert torch.equal(out["top_ids"].cpu().long(), want["top_ids"])
    ref.close(out["logp"], want["logp"], ref.value_tol(want["logp"]), "logp")
    gr, size = ref.logprobs_grad(want, y, 1.0, torch.ones(N), None)
    ref.grad_close(dx, gr, size)


def test_gradient_against_differences(cuda_lib):
    """Central differences of the forward call's own outputs, fp32 logits."""
    N, V, h = 3, 203, 0.05
    x = ref.make_logits(N, V, F32, seed=31, sigma=1.0)
    y = _labels(N, V, 31)
    gl = torch.tensor([1.0, -2.0, 0.5])
    gh = torch.tensor([0.3, 0.7, -1.0])

    def f(z):
        o = cuda_lib.foak_logprobs_forward(z.cuda(), y.cuda())
        return (gl * o["logp"].cpu() + gh * o["entropy"].cpu()).double()

    xd = ref.to_gpu(x)
    o = cuda_lib.foak_logprobs_forward(xd, y.cuda())
    dx, _ = cuda_lib.foak_logprobs_backward(xd, y.cuda(), o["stats"], gl.cuda(), o["entropy"], gh.cuda())
    for j in [0, 1, int(y[0]), int(y[1]), int(y[2]), 100, V - 1]:
        up, dn = x.clone(), x.clone()
        up[:, j] += h
        dn[:, j] -= h
        num = (f(up) - f(dn)) / (2 * h)
        # the outputs' errors over 2 h, and h^2 / 6 times a third derivative below 20
        tol = 3 * (ref.EPS + ref.entropy_tol(V)) / h + h * h / 6 * 20
        assert (num - dx[:, j].cpu().double()).abs().max() < tol


def test_run_out_wait_is_reported(cuda_lib):
    """A copy that is never made ends in the error word, in both launch shapes; the next call is right."""
    ce = cuda_lib
    cases = [ref.make_logits(500, 5000, BF16, seed=1), ref.make_logits(3, 128256, BF16, seed=2)]
    try:
        ce.lib.foak_test_set_wait_limit_ns(100_000_000)
        for x in cases:
            ce.lib.foak_test_skip_row_load(1)
            out = ce.foak_logprobs_forward(ref.to_gpu(x), None, top_k=12)
            torch.cuda.synchronize()
            assert int(out["err"].item()) & ce.FOAK_ERRBIT_TIMEOUT
    finally:
        ce.lib.foak_test_skip_row_load(-1)
        ce.lib.foak_test_set_wait_limit_ns(0)
    for x in cases:
        _check_forward(ce, x, None, 12)
