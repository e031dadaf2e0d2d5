"""The distillation calls against float64: loss, row terms and gradients (fused, in place,
and forward then backward) over types, row shapes, clusters, masks, paddings and repeated
tokens; bounds derived in row_ops_ref."""
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


def _teacher(x, K, T, seed, noise=1.0):
    r = np.random.default_rng(seed + 77)
    z = (x.float() + noise * torch.from_numpy(r.standard_normal(x.shape).astype(np.float32))) / T
    top = z.topk(K, dim=1)
    return top.indices.int(), (top.values - z.logsumexp(1, keepdim=True)).contiguous()


def _check(ce, x, y, ids, t, T=1.0, ce_w=0.0, kd_w=1.0, normalize=True, g=1.0, denom=0.0, modes=("fused", "inplace", "two")):
    want = ref.distill(x, y, ids, t, T, ce_w, kd_w, normalize, g, denom)
    yd = None if y is None else y.cuda()
    idd, td = ids.cuda(), t.cuda()
    how = dict(ce_weight=ce_w, kd_weight=kd_w, temperature=T, normalize=normalize, denom=denom)
    outs = []
    for mode in modes:
        xd = ref.to_gpu(x)
        if mode == "two":
            r = ce.foak_distill_forward(xd, yd, idd, td, want_rows=True, **how)
            go = torch.full((1,), g, device="cuda")
            r["dlogits"], err = ce.foak_distill_backward(xd, yd, idd, td, r["stats"], go, **how)
            assert int(err.item()) == 0
        else:
            keep = xd.clone() if mode == "fused" else None
            dl = ce._dlogits_arg(None, xd, xd.shape[0], xd.shape[1], xd.stride(0) if xd.shape[0] > 1 else max(xd.shape[1], xd.stride(0))) if mode == "fused" else None
            r = ce.foak_distill_fwd_bwd(xd, yd, idd, td, g=g, dlogits=dl, want_rows=True, **how)
            if mode == "fused":
                assert torch.equal(torch.nan_to_num(keep.float()), torch.nan_to_num(xd.float())), "the logits changed"
            else:
                assert r["dlogits"].data_ptr() == xd.data_ptr()
        torch.cuda.synchronize()
        ref.close(r["row_kd"], want["row_kd"], 2 * ref.EPS * want["kd_size"] + 1e-30, f"row_kd ({mode})")
        ref.close(r["row_ce"], want["row_ce"], 2 * ref.EPS * want["ce_size"] + 1e-30, f"row_ce ({mode})")
        loss = torch.tensor([want["loss"]], dtype=torch.float64)
        ref.close(r["loss"], loss, 2 * ref.EPS * (want["loss_size"] if math.isfinite(want["loss_size"]) else 0.0) + 1e-30, f"loss ({mode})")
        ref.grad_close(r["dlogits"], want["dlogits"], want["grad_size"], f"dlogits ({mode})")
        assert int(r["n_valid"].item()) == want["n_valid"] and int(r["err"].item()) == 0
        ign = ~want["ok"]
        if ign.any():
            z = r["dlogits"][ign.cuda()].float()
            assert int(z.count_nonzero()) == 0 and not bool(torch.signbit(z).any())
        outs.append(r)
    return outs, want


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,V,K", [(1, 1, 1), (3, 2, 2), (5, 7, 3), (4, 31, 31), (9, 1000, 64), (6, 8192, 20),
                                   (5, 32000, 256), (3, 50257, 100), (1, 128256, 20), (40, 32000, 20), (90, 50257, 7),
                                   (400, 9001, 50), (170, 128263, 30), (30, 128256, 50), (60, 128263, 30)])
@pytest.mark.parametrize("T,ce_w,normalize", [(1.0, 0.0, True), (1.0, 0.4, False), (2.0, 0.5, True), (0.5, 0.0, False)])
def test_shapes(cuda_lib, dtype, N, V, K, T, ce_w, normalize):
    x = ref.make_logits(N, V, dtype, seed=N + V)
    ids, t = _teacher(x, K, T, N)
    _check(cuda_lib, x, _labels(N, V, N, n_ignore=N // 6), ids, t, T, ce_w, 0.8, normalize, g=0.5)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("ld_more,offset", [(0, 1), (1, 0), (3, 5), (13, 7)])
@pytest.mark.parametrize("N,V", [(7, 5003), (300, 1031), (2, 100001), (30, 100001)])
def test_strides_and_offsets(cuda_lib, dtype, ld_more, offset, N, V):
    x = ref.make_logits(N, V, dtype, seed=V + offset, ld=V + ld_more, offset=offset)
    ids, t = _teacher(x, 12, 1.5, V)
    wide = torch.zeros(N, 20, dtype=torch.int32)
    wide_t = torch.zeros(N, 20)
    wide[:, :12], wide_t[:, :12] = ids, t
    want_ids, want_t = wide[:, :12], wide_t[:, :12]
    y = _labels(N, V, V, n_ignore=1)
    _check(cuda_lib, x, y, ids, t, 1.5, 0.3, 1.0)
    # the teacher's rows as a view of wider ones
    xd = ref.to_gpu(x)
    a = cuda_lib.foak_distill_forward(xd, y.cuda(), ids.cuda(), t.cuda(), temperature=1.5)
    wi, wt = wide.cuda(), wide_t.cuda()
    b = cuda_lib.foak_distill_forward(xd, y.cuda(), wi[:, :12], wt[:, :12], temperature=1.5)
    assert torch.equal(a["loss"], b["loss"]) and torch.equal(a["stats"], b["stats"])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("N,V", [(3, 4099), (200, 4099), (10, 100003)])
def test_padding_repeats_and_the_label(cuda_lib, dtype, normalize, N, V):
    """Padded entries, rows without any entry, -inf entries, repeated tokens, the label among them."""
    K = 9
    x = ref.make_logits(N, V, dtype, seed=6)
    ids, t = _teacher(x, K, 1.0, 6)
    y = _labels(N, V, 6)
    for i in range(N):
        kind = i % 5
        if kind == 0:
            ids[i, 4:] = -1
        elif kind == 1:
            ids[i] = -1
        elif kind == 2:
            t[i, 2:5] = -math.inf
            y[i] = int(ids[i, 0])
        elif kind == 3:
            ids[i, 3] = ids[i, 1]
            ids[i, 7] = ids[i, 1]
            y[i] = int(ids[i, 1])
        else:
            ids[i, :3] = torch.tensor([0, V - 1, 1], dtype=torch.int32)
            y[i] = V - 1
    _check(cuda_lib, x, y, ids, t, 1.0, 0.6, 1.3, normalize)
    _check(cuda_lib, x, y, ids, t, 2.0, 0.6, 1.3, normalize)


def test_teacher_logits_instead_of_log_probabilities(cuda_lib):
    """Renormalised, a row's common shift does not matter; large logits do not overflow."""
    x = ref.make_logits(20, 3001, F32, seed=3)
    ids, t = _teacher(x, 16, 1.0, 3)
    _check(cuda_lib, x, None, ids, t + 500.0, modes=("fused",))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,V", [(6, 32003), (200, 32003), (12, 128259)])
def test_masks(cuda_lib, dtype, N, V):
    low = torch.finfo(dtype).min
    x = ref.make_logits(N, V, dtype, seed=11)
    ids, t = _teacher(x, 10, 1.0, 11)
    y = _labels(N, V, 11)
    for i in range(N):
        away = torch.ones(V, dtype=torch.bool)
        away[ids[i].long()] = False
        away[y[i]] = False
        kind = i % 6
        if kind == 0:
            x[i, away & (torch.arange(V) % 2 == 0)] = -math.inf
        elif kind == 1:
            x[i, away] = low
        elif kind == 2:
            x[i] = low            # a flat row
        elif kind == 3:
            x[i, away] = -math.inf
    _check(cuda_lib, x, y, ids, t, 1.0, 0.5, 1.0)
    _check(cuda_lib, x, y, ids, t, 1.0, 0.0, 1.0)


@pytest.mark.parametrize("V", [1000, 70001])
def test_impossible_targets_give_an_infinite_loss_and_finite_gradients(cuda_lib, V):
    x = ref.make_logits(4, V, F32, seed=12)
    ids, t = _teacher(x, 5, 1.0, 12)
    x[1, ids[1, 2].long()] = -math.inf  # a listed token masked
    x[2] = -math.inf                     # nothing left
    outs, want = _check(cuda_lib, x, None, ids, t)
    assert want["loss"] == math.inf
    for r in outs:
        assert torch.isfinite(r["dlogits"]).all()


def test_nan_stays_in_its_row(cuda_lib):
    N, V = 200, 9000
    x = ref.make_logits(N, V, BF16, seed=13)
    ids, t = _teacher(x, 5, 1.0, 13)
    x[3, 8000] = math.nan
    x[5, 1] = math.inf
    t[7, 1] = math.nan
    r = cuda_lib.foak_distill_fwd_bwd(ref.to_gpu(x), None, ids.cuda(), t.cuda(), want_rows=True)
    dx = r["dlogits"].float().cpu()
    bad = [3, 5, 7]
    keep = [i for i in range(N) if i not in bad]
    assert torch.isnan(dx[bad]).all() and torch.isfinite(dx[keep]).all()
    assert torch.isnan(r["row_kd"].cpu()[bad]).all() and torch.isfinite(r["row_kd"].cpu()[keep]).all()
    assert math.isnan(float(r["loss"]))


def test_denominator_and_weights(cuda_lib):
    x = ref.make_logits(50, 700, F32, seed=14)
    ids, t = _teacher(x, 5, 2.0, 14)
    y = _labels(50, 700, 14, n_ignore=9)
    _check(cuda_lib, x, y, ids, t, 2.0, 0.5, 0.5, denom=1234.0)
    _check(cuda_lib, x, y, ids, t, 2.0, 1.0, 0.0)    # cross-entropy alone
    _check(cuda_lib, x, y, ids, t, 1.0, -0.5, 2.0, g=-3.0)


def test_no_valid_row(cuda_lib):
    x = ref.make_logits(6, 700, BF16, seed=15)
    ids, t = _teacher(x, 5, 1.0, 15)
    y = torch.full((6,), -100)
    r = cuda_lib.foak_distill_fwd_bwd(ref.to_gpu(x), y.cuda(), ids.cuda(), t.cuda())
    assert math.isnan(float(r["loss"])) and int(r["dlogits"].count_nonzero()) == 0 and int(r["n_valid"]) == 0
    e = cuda_lib.foak_distill_fwd_bwd(torch.empty(0, 9, device="cuda"), None, torch.empty(0, 2, dtype=torch.int32, device="cuda"),
                                      torch.empty(0, 2, device="cuda"))
    assert math.isnan(float(e["loss"])) and int(e["err"]) == 0


def test_bad_ids_and_labels_are_reported(cuda_lib):
    x = ref.make_logits(40, 900, F32, seed=16)
    ids, t = _teacher(x, 5, 1.0, 16)
    ids[7, 2] = 900
    want = ref.distill(x, None, ids, t, 1.0, 0.0, 1.0, True)
    xd = ref.to_gpu(x)
    r = cuda_lib.foak_distill_forward(xd, None, ids.cuda(), t.cuda(), want_rows=True)
    assert int(r["err"]) == cuda_lib.FOAK_ERRBIT_LABEL_RANGE
    ref.close(r["row_kd"], want["row_kd"], 2 * ref.EPS * want["kd_size"], "row_kd")
    dx, _ = cuda_lib.foak_distill_backward(xd, None, ids.cuda(), t.cuda(), r["stats"])
    ref.grad_close(dx, want["dlogits"], want["grad_size"])
    ids[7, 2] = -1
    y = _labels(40, 900, 16)
    y[9] = 900
    r = cuda_lib.foak_distill_fwd_bwd(xd, y.cuda(), ids.cuda(), t.cuda())
    assert int(r["err"]) == cuda_lib.FOAK_ERRBIT_LABEL_RANGE and int(r["n_valid"]) == 39
    assert int(r["dlogits"][9].count_nonzero()) == 0


def test_offsets_past_32_bits(cuda_lib):
    V, N = 40_009, 60_001
    x = torch.zeros(N, V, dtype=BF16, device="cuda")
    row = ref.make_logits(1, V, BF16, seed=4)
    x[N - 1] = row[0].cuda()
    ids, t = _teacher(row, 6, 1.0, 4)
    ids_all = torch.full((N, 6), -1, dtype=torch.int32, device="cuda")
    t_all = torch.zeros(N, 6, device="cuda")
    ids_all[N - 1], t_all[N - 1] = ids[0].cuda(), t[0].cuda()
    y = torch.full((N,), -100, dtype=torch.int64, device="cuda")
    y[N - 1] = 77
    want = ref.distill(row, torch.tensor([77]), ids, t, 1.0, 0.5, 1.0, True)
    r = cuda_lib.foak_distill_fwd_bwd(x, y, ids_all, t_all, ce_weight=0.5)
    ref.grad_close(r["dlogits"][N - 1:], want["dlogits"], want["grad_size"])
    assert int(r["dlogits"][: N - 1].count_nonzero()) == 0


def test_same_bits_again_and_in_a_graph(cuda_lib):
    N, V, K = 300, 32005, 30
    x = ref.make_logits(N, V, BF16, seed=17)
    ids, t = (a.cuda() for a in _teacher(x, K, 1.0, 17))
    y = _labels(N, V, 17, n_ignore=20).cuda()
    xd = ref.to_gpu(x)
    how = dict(ce_weight=0.5, temperature=2.0)
    dl = cuda_lib._dlogits_arg(None, xd, N, V, V)
    a = cuda_lib.foak_distill_fwd_bwd(xd, y, ids, t, dlogits=dl, **how)
    a_loss, a_dl = a["loss"].clone(), dl.clone()
    ws = torch.zeros(cuda_lib.foak_ce_workspace_size(N), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    dl.zero_()
    with torch.cuda.graph(g, stream=side):
        b = cuda_lib.foak_distill_fwd_bwd(xd, y, ids, t, dlogits=dl, workspace_tensor=ws, **how)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a_loss, b["loss"]) and torch.equal(a_dl, dl)


def test_gradient_against_differences(cuda_lib):
    N, V, K, h = 3, 203, 11, 0.05
    x = ref.make_logits(N, V, F32, seed=31, sigma=1.0)
    y = _labels(N, V, 31)
    ids, t = _teacher(x, K, 2.0, 31)
    how = dict(ce_weight=0.7, kd_weight=1.5, temperature=2.0, normalize=False)

    def f(z):
        o = cuda_lib.foak_distill_forward(z.cuda(), y.cuda(), ids.cuda(), t.cuda(), want_rows=True, **how)
        return (0.7 * o["row_ce"].cpu().double() + 1.5 * o["row_kd"].cpu().double()) / N

    r = cuda_lib.foak_distill_fwd_bwd(ref.to_gpu(x), y.cuda(), ids.cuda(), t.cuda(), **how)
    for j in [0, int(y[0]), int(y[1]), int(ids[0, 0]), int(ids[1, 3]), 100, V - 1]:
        up, dn = x.clone(), x.clone()
        up[:, j] += h
        dn[:, j] -= h
        num = (f(up) - f(dn)) / (2 * h)
        tol = 3 * 10 * ref.EPS / h + h * h / 6 * 3  # the rows' errors over 2 h; a third derivative below 3
        assert (num - r["dlogits"][:, j].cpu().double()).abs().max() < tol


def test_run_out_wait_is_reported(cuda_lib):
    ce = cuda_lib
    cases = [ref.make_logits(500, 5000, BF16, seed=1), ref.make_logits(3, 128256, BF16, seed=2)]
    try:
        ce.lib.foak_test_set_wait_limit_ns(100_000_000)
        for x in cases:
            ids, t = _teacher(x, 5, 1.0, 1)
            ce.lib.foak_test_skip_row_load(1)
            r = ce.foak_distill_fwd_bwd(ref.to_gpu(x), None, ids.cuda(), t.cuda())
            torch.cuda.synchronize()
            assert int(r["err"]) & ce.FOAK_ERRBIT_TIMEOUT
    finally:
        ce.lib.foak_test_skip_row_load(-1)
        ce.lib.foak_test_set_wait_limit_ns(0)
    for x in cases:
        ids, t = _teacher(x, 5, 1.0, 1)
        _check(ce, x, None, ids, t)
