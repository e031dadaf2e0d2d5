"""Ends of the ranges that the log-probability and distillation calls take: temperatures from
2^-19 to 2^19, logits far from 0, rows of millions of elements, outputs left out, bad ids; bounds
as in row_ops_ref.

Gradients get one absolute term more than there: an exponential below the least normal float,
2^-126, is 0, and the gradient has it times the weights over the temperature."""
import math

import numpy as np
import pytest
import torch

import row_ops_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
LEAST = 2.0 ** -126
TEMPERATURES = (2.0 ** -19, 2.0 ** -10, 2.0 ** 10, 2.0 ** 19)


def _labels(N, V, seed):
    return torch.from_numpy(np.random.default_rng(seed + 1000).integers(0, V, N))


def _far_rows(V, dtype):
    """Logits at which the exponents of one temperature, of both or of none are far apart."""
    base = ref.make_logits(7, V, F32, seed=V)
    x = torch.empty(7, V, dtype=dtype)
    x[0] = base[0]
    x[1] = base[1] + 800
    x[2] = base[2] - 5000
    x[3] = base[3] * 1e-3 + 20
    x[4] = base[4] * 1e4 + 2e9
    x[5] = base[5] * 1e8
    x[6] = base[6] * 100 - 3e9
    return x


def _close_gradient(got, want, size, flushed):
    tol = ref.HALF_STEP[got.dtype] * want.abs() * 1.0001 + 4 * ref.EPS * size + flushed + 1e-37
    ref.close(got, want, tol, "dlogits")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [1201, 100003])
@pytest.mark.parametrize("T", TEMPERATURES)
@pytest.mark.parametrize("ce_w", [0.5, 0.0])
def test_distillation_at_far_exponents(cuda_lib, dtype, V, T, ce_w):
    """The cross-entropy part has temperature 1 whatever T is."""
    ce = cuda_lib
    x = _far_rows(V, dtype)
    N, K, kd_w = x.shape[0], 8, 0.8
    r = np.random.default_rng(V)
    z = (x.double() + torch.from_numpy(r.standard_normal((N, V)))) / T
    top = z.topk(K, dim=1)
    ids, t = top.indices.int(), (top.values - z.logsumexp(1, keepdim=True)).float()
    y = _labels(N, V, 3)
    y[::2] = x.float().argmax(1)[::2]
    want = ref.distill(x, y, ids, t, T, ce_w, kd_w, True)
    flushed = LEAST * (abs(ce_w) + kd_w / T) / N
    how = dict(ce_weight=ce_w, kd_weight=kd_w, temperature=T)
    xd = ref.to_gpu(x)
    a = ce.foak_distill_fwd_bwd(xd.clone(), y.cuda(), ids.cuda(), t.cuda(), want_rows=True, **how)
    b = ce.foak_distill_forward(xd, y.cuda(), ids.cuda(), t.cuda(), want_rows=True, **how)
    b["dlogits"], _ = ce.foak_distill_backward(xd, y.cuda(), ids.cuda(), t.cuda(), b["stats"], **how)
    for out in (a, b):
        ref.close(out["row_ce"], want["row_ce"], 2 * ref.EPS * want["ce_size"] + 1e-30, "row_ce")
        ref.close(out["row_kd"], want["row_kd"], 2 * ref.EPS * want["kd_size"] + 1e-30, "row_kd")
        _close_gradient(out["dlogits"], want["dlogits"], want["grad_size"], flushed)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [1201, 100003])
@pytest.mark.parametrize("T", TEMPERATURES)
def test_log_probabilities_at_far_exponents(cuda_lib, dtype, V, T):
    ce = cuda_lib
    x = _far_rows(V, dtype)
    N, K = x.shape[0], 9
    y = _labels(N, V, 4)
    y[::2] = x.float().argmax(1)[::2]
    want = ref.logprobs(x, y, K, T)
    xd = ref.to_gpu(x)
    out = ce.foak_logprobs_forward(xd, y.cuda(), top_k=K, temperature=T)
    for k in ("lse", "logp", "top_logprobs"):
        ref.close(out[k], want[k], ref.value_tol(want[k]), k)
    ref.close(out["entropy"], want["entropy"], ref.entropy_tol(V), "entropy")
    ref.tops_equal(out["top_ids"], want["top_ids"])
    gl, gh = torch.linspace(-1, 1, N), torch.linspace(0.5, -0.7, N)
    dx, _ = ce.foak_logprobs_backward(xd, y.cuda(), out["stats"], gl.cuda(), out["entropy"], gh.cuda(), temperature=T)
    g, size = ref.logprobs_grad(want, y, T, gl, gh)
    # p (ln p + H) of a flushed p has a factor up to 126 ln 2 + ln V more
    _close_gradient(dx, g, size, 101 * LEAST / T)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,V,K", [(1, 1, 1), (5, 7, 0), (7, 8192, 20), (3, 50257, 0), (2, 128263, 40), (300, 4099, 0),
                                   (200, 40001, 17), (64, 128256, 0)])
def test_without_the_entropy(cuda_lib, dtype, N, V, K):
    """want_entropy=False and no other output: the same values, masks and infinities among them."""
    low = torch.finfo(dtype).min
    x = ref.make_logits(N, V, dtype, seed=N + V)
    r = np.random.default_rng(7)
    for i in range(N):
        drop = torch.from_numpy(r.random(V) < 0.5)
        kind = i % 8
        if kind == 1:
            x[i, drop] = -math.inf
        elif kind == 2:
            x[i, drop] = low
        elif kind == 3:
            x[i] = -math.inf
        elif kind == 4:
            x[i] = low
        elif kind == 5:
            x[i] = x[i] * 1e30
        elif kind == 6:
            x[i] = -math.inf
            x[i, drop] = low
    y = _labels(N, V, 8)
    y[N // 3::11] = -100
    T = 0.7 if V % 2 else 1.0
    want = ref.logprobs(x, y, K, T)
    for k in ("lse", "logp"):  # the lowest value over T < 1 is out of float32's range
        want[k] = want[k].float().double()
    xd = ref.to_gpu(x)
    out = cuda_lib.foak_logprobs_forward(xd, y.cuda(), top_k=K, temperature=T, want_entropy=False)
    assert out["entropy"] is None
    keys = ("lse", "logp") + (("top_logprobs",) if K else ())
    for k in keys:
        ref.close(out[k], want[k], ref.value_tol(want[k]), k)
    if K:
        ref.tops_equal(out["top_ids"], want["top_ids"])
    gl = torch.linspace(-1, 1, N)
    dx, _ = cuda_lib.foak_logprobs_backward(xd, y.cuda(), out["stats"], gl.cuda(), temperature=T)
    ref.grad_close(dx, *ref.logprobs_grad(want, y, T, gl, None))
    only = cuda_lib.foak_logprobs_forward(xd, y.cuda(), top_k=K, temperature=T, want_entropy=False, want_lse=False,
                                          want_stats=False)
    assert only["lse"] is None and only["stats"] is None and torch.equal(only["logp"], out["logp"])
    # every row, and no output at all but the top tokens
    want = ref.logprobs(x, None, K, T)
    out = cuda_lib.foak_logprobs_forward(xd, None, top_k=K, temperature=T, want_entropy=False)
    want["lse"] = want["lse"].float().double()
    ref.close(out["lse"], want["lse"], ref.value_tol(want["lse"]), "lse")
    if K:
        ref.tops_equal(out["top_ids"], want["top_ids"])


def test_without_the_entropy_nan_stays_in_its_row(cuda_lib):
    for dtype in (BF16, F32):
        for N, V, K in ((5, 33000, 0), (5, 128256, 6)):
            x = ref.make_logits(N, V, dtype, seed=2)
            x[1, 20000], x[3, 31] = math.nan, math.inf
            out = cuda_lib.foak_logprobs_forward(ref.to_gpu(x), None, top_k=K, want_entropy=False)
            assert torch.isnan(out["lse"]).tolist() == [False, True, False, True, False]


# Rows with a logit 0 at every 64th place and a logit c at the others: every warp's maximum is 0
# soon, and a thread adds the same number again and again.  A chain of float32 additions of one
# number rounds the same way for long: 4096 of them may lose 5e-5 (at c = -0.369), 3e-5 (-0.898).
FLAT = (-0.369140625, -0.8984375, -0.400390625)


def _flat(V, c):
    """ln S, entropy and the probabilities of a logit 0 and of a logit c."""
    e, n = math.exp(c), (V + 63) // 64
    s = n + (V - n) * e
    return math.log(s), math.log(s) - (V - n) * e * c / s, 1 / s, e / s


def _fill_flat(row, c):
    row.fill_(c)
    row[::64] = 0.0


@pytest.mark.parametrize("dtype,V", [(F32, 134_217_733), (BF16, 268_435_471), (BF16, 2 ** 31 - 1)])
def test_sums_of_very_long_rows(cuda_lib, dtype, V):
    ce = cuda_lib
    x = torch.empty(1, V, dtype=dtype, device="cuda")
    y = torch.tensor([64 * 1001], device="cuda")
    for c in FLAT if V < 2 ** 30 else FLAT[:1]:
        _fill_flat(x[0], c)
        ln_s, h, p0, pc = _flat(V, c)
        for entropy in (True, False):
            out = ce.foak_logprobs_forward(x, y, want_entropy=entropy)
            tol = ref.EPS + 6 * ref.U * ln_s
            assert abs(float(out["lse"]) - ln_s) < tol and abs(float(out["logp"]) + ln_s) < tol
            if entropy:
                assert abs(float(out["entropy"]) - h) < ref.entropy_tol(V)
        out = ce.foak_distill_forward(x, y, y[:, None].int(), torch.zeros(1, 1, device="cuda"), ce_weight=1.0,
                                      temperature=2.0, want_rows=True)
        assert abs(float(out["row_ce"]) - ln_s) < 2 * ref.EPS * (1 + ln_s)
        assert abs(float(out["row_kd"]) - _flat(V, c / 2)[0]) < 2 * ref.EPS * (1 + ln_s)


def test_sums_of_long_rows_that_a_cta_has_to_itself(cuda_lib):
    """More rows than clusters take, most of them ignored."""
    ce = cuda_lib
    N, V, K = 160, 16_777_221, 1
    x = torch.zeros(N, V, dtype=F32, device="cuda")
    y = torch.full((N,), -100, device="cuda")
    ids, t = torch.zeros(N, K, dtype=torch.int32, device="cuda"), torch.zeros(N, K, device="cuda")
    rows = (0, 70, 159)
    cs = FLAT
    for i, c in zip(rows, cs):
        _fill_flat(x[i], c)
        y[i] = 64
        ids[i] = 6
    out = ce.foak_logprobs_forward(x, y)
    two = ce.foak_distill_forward(x, y, ids, t, ce_weight=0.5, temperature=2.0, want_rows=True)
    one = ce.foak_distill_forward(x, y, ids, t, ce_weight=0.5, want_rows=True)
    g2 = ce.foak_distill_fwd_bwd(x, y, ids, t, ce_weight=0.5, temperature=2.0, want_rows=True,
                                 dlogits=torch.empty_like(x))
    for i, c in zip(rows, cs):
        ln_1, h, p0, pc = _flat(V, c)
        ln_2, _, q0, qc = _flat(V, c / 2)
        tol = 2 * ref.EPS * (1 + ln_1)
        assert abs(float(out["lse"][i]) - ln_1) < ref.EPS + 6 * ref.U * ln_1
        assert abs(float(out["entropy"][i]) - h) < ref.entropy_tol(V)
        assert abs(float(one["row_ce"][i]) - ln_1) < tol and abs(float(one["row_kd"][i]) - (ln_1 - c)) < tol
        for r in (two, g2):
            assert abs(float(r["row_ce"][i]) - ln_1) < tol and abs(float(r["row_kd"][i]) - (ln_2 - c / 2)) < tol
        size = (0.5 * pc + 0.5 * qc) / 3
        far = g2["dlogits"][i, 7:64].double()
        assert float((far - size).abs().max()) < (4 * ref.EPS + ref.HALF_STEP[F32]) * size
    g1 = ce.foak_distill_fwd_bwd(x, y, ids, t, ce_weight=0.5)  # in place
    for i, c in zip(rows, cs):
        size = 1.5 * _flat(V, c)[3] / 3
        far = g1["dlogits"][i, 7:64].double()
        assert float((far - size).abs().max()) < (4 * ref.EPS + ref.HALF_STEP[F32]) * size


@pytest.mark.parametrize("N,V", [(40, 900), (3, 70001), (700, 1031)])
def test_a_bad_teacher_id_is_reported_by_every_call(cuda_lib, N, V):
    """By the backward call too, whichever rows it is in; the next call's word is clean again."""
    ce = cuda_lib
    x = ref.make_logits(N, V, F32, seed=16)
    r = np.random.default_rng(1)
    ids = torch.from_numpy(np.stack([r.permutation(V)[:5] for _ in range(N)])).int()
    t = torch.log_softmax(torch.from_numpy(r.standard_normal((N, 5))), 1).float()
    xd, td = ref.to_gpu(x), t.cuda()
    for row in (0, N // 2, N - 1):
        bad = ids.clone()
        bad[row, 2] = V + 3 * row
        want = ref.distill(x, None, bad, t, 1.0, 0.0, 1.0, True)
        f = ce.foak_distill_forward(xd, None, bad.cuda(), td)
        dx, err = ce.foak_distill_backward(xd, None, bad.cuda(), td, f["stats"])
        both = ce.foak_distill_fwd_bwd(xd.clone(), None, bad.cuda(), td)
        assert int(f["err"]) == int(both["err"]) == int(err) == ce.FOAK_ERRBIT_LABEL_RANGE
        ref.grad_close(dx, want["dlogits"], want["grad_size"])
        # not of a row that does not count
        y = torch.zeros(N, dtype=torch.int64)
        y[row] = -100
        f = ce.foak_distill_forward(xd, y.cuda(), bad.cuda(), td)
        _, err = ce.foak_distill_backward(xd, y.cuda(), bad.cuda(), td, f["stats"])
        assert int(f["err"]) == int(err) == 0
        y[0 if row else 1] = V
        _, err = ce.foak_distill_backward(xd, y.cuda(), bad.cuda(), td, f["stats"])
        assert int(err) == ce.FOAK_ERRBIT_LABEL_RANGE
    _, err = ce.foak_distill_backward(xd, None, ids.cuda(), td, f["stats"])
    assert int(err) == 0


def test_a_denominator_that_is_no_number_is_none(cuda_lib):
    """denom > 0, else the number of valid rows: for every place of the gradient."""
    ce = cuda_lib
    N, V = 400, 1031
    x = ref.make_logits(N, V, F32, seed=5)
    y = _labels(N, V, 5)
    y[::3] = -100
    ids = torch.arange(N * 4, dtype=torch.int32).reshape(N, 4) % V
    t = torch.log_softmax(torch.from_numpy(np.random.default_rng(2).standard_normal((N, 4))), 1).float()
    xd, yd, idd, td = ref.to_gpu(x), y.cuda(), ids.cuda(), t.cuda()
    how = dict(ce_weight=0.5)
    a = ce.foak_distill_fwd_bwd(xd.clone(), yd, idd, td, **how)
    b = ce.foak_distill_fwd_bwd(xd.clone(), yd, idd, td, denom=math.nan, **how)
    assert torch.equal(a["loss"], b["loss"]) and torch.equal(a["dlogits"], b["dlogits"])
    f = ce.foak_distill_forward(xd, yd, idd, td, **how)
    c, _ = ce.foak_distill_backward(xd, yd, idd, td, f["stats"], **how)
    d, _ = ce.foak_distill_backward(xd, yd, idd, td, f["stats"], denom=math.nan, **how)
    assert torch.equal(c, d)


@pytest.mark.parametrize("per_sm", [2, 4, 6])
@pytest.mark.parametrize("V,K", [(4099, 30), (1031, 200)])
def test_a_few_rows_a_cta(cuda_lib, per_sm, V, K):
    """The scale of every row is that of all rows, whichever closing warp takes it and however many rows a CTA
    has: with two, one closing warp is done while the other has its row still before it."""
    ce = cuda_lib
    N = per_sm * torch.cuda.get_device_properties(0).multi_processor_count
    x = ref.make_logits(N, V, BF16, seed=N)
    ids = torch.from_numpy(np.random.default_rng(N).integers(0, V, (N, K))).int()
    t = torch.log_softmax(torch.from_numpy(np.random.default_rng(N + 1).standard_normal((N, K))), 1).float()
    want = ref.distill(x, None, ids, t, 2.0, 0.0, 1.0, True, g=0.25)
    xd = ref.to_gpu(x)
    for _ in range(5):
        out = ce.foak_distill_fwd_bwd(xd.clone(), None, ids.cuda(), t.cuda(), temperature=2.0, g=0.25)
        assert int(out["n_valid"]) == N
        ref.grad_close(out["dlogits"], want["dlogits"], want["grad_size"])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_about_the_borders_of_the_cluster_sizes(cuda_lib, dtype):
    """8, 4, 2 and 1 CTAs a row as the rows get more: the largest number of rows at each size, and one more."""
    ce = cuda_lib
    sms, V, K = torch.cuda.get_device_properties(0).multi_processor_count, 100_003, 7
    most = 2 * sms + 1
    x = ref.make_logits(1, V, dtype, seed=1).repeat(most, 1)
    x[0, torch.arange(1, K + 1) * 13_001] = 17.0 - torch.arange(K).to(dtype)  # no ties, whose order a turn would change
    for i in range(most):  # rows that differ in a known way: a turn of one row
        x[i] = torch.roll(x[0], i)
    y = (torch.arange(most) * 7) % V
    want = ref.logprobs(x[:1], None, K, 1.0)
    lnp, top = want["lnp"][0], want["top_ids"][0]
    assert len(set(x[0, top].tolist())) == K
    xd, yd = ref.to_gpu(x), y.cuda()
    ids = torch.stack([(top + i) % V for i in range(most)])
    t = want["top_logprobs"].float().expand(most, K).contiguous().cuda()
    logp = torch.stack([lnp[(y[i] - i) % V] for i in range(most)])
    kd = ref.distill(x[:1], None, ids[:1].int(), t[:1].cpu(), 1.0, 0.0, 1.0, True)
    for at_most in (2 * sms, sms):
        for k in (8, 4, 2, 1):
            for N in sorted({max(1, at_most // k), at_most // k + 1, 1}):
                out = ce.foak_logprobs_forward(xd[:N], yd[:N], top_k=K)
                ref.tops_equal(out["top_ids"], ids[:N])
                ref.close(out["logp"], logp[:N], ref.value_tol(logp[:N]), "logp")
                out = ce.foak_logprobs_forward(xd[:N], yd[:N])
                ref.close(out["lse"], want["lse"].expand(N), ref.value_tol(want["lse"]).expand(N), "lse")
                idd = ids[:N].int().cuda()
                f = ce.foak_distill_forward(xd[:N], None, idd, t[:N], want_rows=True)
                b = ce.foak_distill_fwd_bwd(xd[:N], None, idd, t[:N], want_rows=True, dlogits=torch.empty_like(xd[:N]))
                for r in (f, b):
                    ref.close(r["row_kd"], kd["row_kd"].expand(N), 2 * ref.EPS * kd["kd_size"].expand(N) + 1e-30, "row_kd")
