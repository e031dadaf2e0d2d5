"""Float64 references of the log-probability and distillation calls, and the bounds of
their errors.

Bounds.  u = 2^-24 is half a float32 step.  A kernel's exponent (x - m) c carries a few
u relative, its exponential 2^-22 relative; a row's sum adds at most about a hundred
roundings one after another (a thread's partial sums, rescalings at a new maximum, the
joining tree).  So ln S is off by at most 2^-22 + (30 + 100 + 4 * 10) u < 1.1e-5 =: EPS,
a log probability by EPS and a few u of its own size, an entropy (ln S minus a weighted
mean of exponents up to ln S + H) by 2 EPS (1 + ln V), a probability by 2 EPS relative.
Gradients are sums of a few such terms; each is bounded by 4 EPS times the sum of the
terms' sizes, plus half a step of the storage type (2^-8 bf16, 2^-24 fp32).
"""
import math

import numpy as np
import torch

EPS = 1.1e-5
U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def softmax_parts(x, T):
    """(max, (x - max) / T, p, ln S) in float64; p is 0 in a row of -inf alone."""
    m = x.max(dim=1, keepdim=True).values
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    d = (x - m) / T
    s = d.exp().sum(1, keepdim=True)
    p = torch.where(s == 0, torch.zeros_like(d), d.exp() / s)
    return m, d, p, s.log()


def logprobs(logits, labels, K, T, ignore_index=-100):
    x = logits.detach().cpu().double()
    N, V = x.shape
    y = None if labels is None else labels.cpu()
    ok = torch.ones(N, dtype=torch.bool) if y is None else (y != ignore_index) & (y >= 0) & (y < V)
    m, d, p, ln_s = softmax_parts(x, T)
    nan = torch.isnan(ln_s[:, 0])
    lnp = torch.where(ln_s == -math.inf, torch.full_like(d, -math.inf), d - ln_s)
    out = {"ok": ok, "lnp": lnp, "p": p, "ln_s": ln_s[:, 0], "size": d.abs()}
    out["lse"] = torch.where(ok, (m / T + ln_s)[:, 0], 0.0)
    out["entropy"] = torch.where(ok & ~nan, -torch.xlogy(p, p).sum(1), torch.where(ok, math.nan, 0.0))
    if y is not None:
        out["logp"] = torch.where(ok, lnp.gather(1, y.clamp(0, V - 1)[:, None])[:, 0], 0.0)
    if K:
        order = torch.sort(x + 0.0, dim=1, descending=True, stable=True).indices[:, :K]
        out["top_ids"] = torch.where((ok & ~nan)[:, None], order, -1)
        out["top_logprobs"] = torch.where(ok[:, None], torch.where(nan[:, None], math.nan, lnp.gather(1, order)), 0.0)
    return out


def logprobs_grad(ref, labels, T, gl, gh):
    """Gradient and the sum of its terms' sizes."""
    p, lnp, ok = ref["p"], ref["lnp"].clamp(min=-1e30), ref["ok"]
    N, V = p.shape
    gl = (torch.zeros(N) if gl is None else gl.cpu()).double()[:, None] / T
    gh = (torch.zeros(N) if gh is None else gh.cpu()).double()[:, None] / T
    one = torch.zeros_like(p)
    y = labels.cpu().clamp(0, V - 1)
    one[torch.arange(N), y] = 1.0
    h = torch.where(ok, ref["entropy"], 0.0)[:, None]
    dx = gl * (one - p) - gh * p * (lnp + h)
    size = gl.abs() * (one + p) + gh.abs() * p * (lnp.abs() + h.abs() + 1)
    zero = torch.zeros_like(dx)
    return torch.where(ok[:, None], dx, zero), torch.where(ok[:, None], size, zero)


def distill(logits, labels, ids, t, T, ce_w, kd_w, normalize, g=1.0, denom=0.0, ignore_index=-100):
    x = logits.detach().cpu().double()
    N, V = x.shape
    y = None if labels is None else labels.cpu()
    ok = torch.ones(N, dtype=torch.bool) if y is None else (y != ignore_index) & (y >= 0) & (y < V)
    D = denom if denom > 0 else float(ok.sum())
    ids, t = ids.cpu().long(), t.cpu().double()
    there = (ids >= 0) & (ids < V)
    at = ids.clamp(0, V - 1)
    q = torch.where(there, t.exp(), 0.0)
    if normalize:
        tt = torch.where(there, t, -math.inf)
        top = tt.max(1, keepdim=True).values
        e = torch.where(tt == -math.inf, 0.0, (tt - top).exp())
        tot = e.sum(1, keepdim=True)
        q = torch.where(tot > 0, e / tot, 0.0)
    m, d, p, ln_s = softmax_parts(x, T)
    m1, d1, p1, ln_s1 = softmax_parts(x, 1.0)
    lnp = torch.where(ln_s == -math.inf, torch.full_like(d, -math.inf), d - ln_s)
    lnp1 = torch.where(ln_s1 == -math.inf, torch.full_like(d, -math.inf), d1 - ln_s1)
    terms = torch.where(q > 0, torch.xlogy(q, q) - q * lnp.gather(1, at), torch.zeros_like(q))
    kd = terms.sum(1)
    kd_size = torch.where(q > 0, q * (1 + q.log().abs() + lnp.gather(1, at).abs() + t.abs()), torch.zeros_like(q)).sum(1)
    ce = torch.zeros(N, dtype=torch.float64)
    ce_size = torch.zeros(N, dtype=torch.float64)
    yy = None if y is None else y.clamp(0, V - 1)[:, None]
    if ce_w != 0:
        ce = -lnp1.gather(1, yy)[:, 0]
        ce_size = 1 + ce.abs()
    kd, ce = torch.where(ok, kd, 0.0), torch.where(ok, ce, 0.0)
    out = {"ok": ok, "row_kd": kd, "row_ce": ce, "kd_size": torch.where(ok, kd_size, 0.0), "ce_size": torch.where(ok, ce_size, 0.0)}
    rows = (ce_w * ce if ce_w else 0.0) + (kd_w * kd if kd_w else torch.zeros_like(kd))
    sizes = abs(ce_w) * out["ce_size"] + abs(kd_w) * out["kd_size"]
    out["loss"] = float(rows.sum() / D) if D else math.nan
    out["loss_size"] = float(sizes.sum() / D) if D else math.nan
    scale = g / D if D else 0.0
    dx = kd_w / T * q.sum(1, keepdim=True) * p
    size = dx.abs()
    flat = (torch.arange(N)[:, None] * V + at).reshape(-1)
    dx.view(-1).index_add_(0, flat, (-kd_w / T * q).reshape(-1))
    size.view(-1).index_add_(0, flat, (abs(kd_w) / T * q).reshape(-1))
    if ce_w != 0:
        dx += ce_w * p1
        size += abs(ce_w) * p1
        dx[torch.arange(N), yy[:, 0]] -= ce_w
        size[torch.arange(N), yy[:, 0]] += abs(ce_w)
    zero = torch.zeros_like(dx)
    out["dlogits"] = torch.where(ok[:, None], dx * scale, zero)
    out["grad_size"] = torch.where(ok[:, None], size * abs(scale), zero)
    out["n_valid"] = int(ok.sum())
    return out


def close(got, ref, tol, what):
    """got (a tensor) within tol of ref; NaN and infinities have to be equal."""
    got = got.detach().cpu().double()
    tol = torch.as_tensor(tol, dtype=torch.float64).expand_as(ref)
    same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    err = (got - ref).abs()
    bad = ~same & ~(err <= tol)
    if bad.any():
        i = tuple(int(k) for k in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {i}: got {float(got[i])!r}, "
                             f"reference {float(ref[i])!r}, tolerance {float(tol[i]):.3g}")


def tops_equal(got, want):
    """The top tokens' ids (int32, on the GPU or not) are the reference's, in its order."""
    assert got.dtype == torch.int32 and got.shape == want.shape
    got = got.detach().cpu().long()
    off = (got != want).any(1)
    assert not off.any(), f"top ids of {int(off.sum())} rows: {got[off][:2]}, reference {want[off][:2]}"


def grad_close(got, ref, size, what="dlogits"):
    half = HALF_STEP[got.dtype]
    # 1e-37: an exponential below the least normal float is 0
    close(got, ref, half * ref.abs() * 1.0001 + 4 * EPS * size + 1e-37, what)


def value_tol(ref, T=1.0):
    """Of a log probability or log-sum-exp: EPS, and a few roundings of its own size."""
    return EPS + 6 * U * torch.nan_to_num(ref.abs(), nan=0.0, posinf=0.0, neginf=0.0)


def entropy_tol(V):
    return 2 * EPS * (1 + math.log(max(V, 2)))


def make_logits(N, V, dtype, seed, ld=None, offset=0, sigma=2.0):
    """N x V logits on the CPU in `dtype`, a view with row stride ld and a start offset (elements)."""
    ld = V if ld is None else ld
    r = np.random.default_rng(seed)
    buf = torch.zeros(N * ld + offset, dtype=dtype)
    x = buf[offset:].as_strided((N, V), (ld, 1))
    a = r.standard_normal((N, V)) * sigma
    hot = r.integers(0, V, (N, 3))
    np.put_along_axis(a, hot, 6 + 6 * r.random((N, 3)), axis=1)
    x.copy_(torch.from_numpy(a))
    return x


def to_gpu(x):
    """The same view (strides, offset modulo 16 bytes) on the GPU."""
    es = x.element_size()
    off = x.storage_offset()
    n = off + ((x.shape[0] - 1) * x.stride(0) + x.shape[1] if x.numel() else 0)
    buf = torch.zeros(max(n, 1), dtype=x.dtype, device="cuda")
    v = buf.as_strided(x.shape, x.stride(), off)
    v.copy_(x)
    assert (v.data_ptr() - buf.data_ptr()) == off * es
    return v
