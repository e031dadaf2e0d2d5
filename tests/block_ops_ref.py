"""64-bit references of the residual norms, rotary positions and the paged cache, with bounds.

A bound counts the roundings of float32 arithmetic (U = 2^-24, half a step relative to a value)
along the longest chain of operations that a result goes through; the storage type's own
rounding, half a step of the result, is added where results are compared.  Sums over a row
are at most CHAIN additions deep: 64 by a thread (32768 elements by 512 threads), then two
trees of 5, and a few products; a sum over N rows N / 128 by a group and then 16 + 32.
"""
import math

import torch

U = 2.0 ** -24
CHAIN = 80
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def row_chain(N):
    return N / 128 + 60


def assert_close(got, want, what):
    """``want`` is (value, bound) in 64 bits; got within the bound and half a step of its type."""
    ref, tol = want
    g = got.detach().cpu().double().reshape(ref.shape)
    half = 0.0 if got.dtype == torch.float64 else torch.finfo(got.dtype).eps / 2
    off = (g - ref).abs()
    room = tol + half * (ref.abs() + tol) + 1e-37
    bad = ~(off <= room)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off by up to {float((off / room).nan_to_num(9e9).max()):.3g} bounds"


def make_norm(N, D, dtype, gate, post, seed, cancel=False):
    """CPU tensors of a residual norm in ``dtype``: dict(X, R, gamma, post_gamma, gate, dY, dH)."""
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]

    def n(*shape):
        return torch.randn(*shape, generator=g)

    X, R = n(N, D), n(N, D) * n(D).exp()
    if cancel:
        R = -X + 0.01 * n(N, D)
    gates = {"none": None, "channel": n(D), "row": n(N, 1), "full": n(N, D)}
    out = dict(X=X, R=R, gamma=1 + 0.3 * n(D), post_gamma=1 + 0.3 * n(D) if post else None, gate=gates[gate], dY=n(N, D), dH=n(N, D))
    return {k: None if v is None else v.to(dt) for k, v in out.items()}


def _d(t):
    return None if t is None else t.detach().cpu().double()


def norm_forward(X, R, gamma, gate, post_gamma, scale, eps, post_eps):
    """{name: (value, bound)} of H, Y, rstd, post_rstd."""
    X, R, gamma, gate, post_gamma = _d(X), _d(R), _d(gamma), _d(gate), _d(post_gamma)
    out, E = {}, (CHAIN / 2 + 6) * U  # of an inverse root: half the sum's error, and the root's two steps
    u = X
    if post_gamma is not None:
        r1 = 1 / (X.square().mean(1, keepdim=True) + post_eps).sqrt()
        out["post_rstd"] = (r1[:, 0], r1[:, 0] * E)
        u = X * r1 * post_gamma
    add = scale * u * (1.0 if gate is None else gate)
    h = R + add
    dh = add.abs() * (E + 6 * U) + (h.abs() + add.abs()) * U
    out["H"] = (h, dh)
    if gamma is not None:
        ms = h.square().mean(1, keepdim=True) + eps
        r = 1 / ms.sqrt()
        dr = E + (h.abs() * dh).mean(1, keepdim=True) / ms
        out["rstd"] = (r[:, 0], (r * dr)[:, 0])
        out["Y"] = (h * r * gamma, (h * r * gamma).abs() * (dr + 4 * U) + dh * (r * gamma).abs())
    return out


def norm_backward(dY, dH, H, rstd, gamma, X, gate, post_gamma, post_rstd, scale):
    """{name: (value, bound)} of dR, dX, dgamma, dgate, dpost_gamma."""
    dY, dH, H, gamma, X, gate, post_gamma = _d(dY), _d(dH), _d(H), _d(gamma), _d(X), _d(gate), _d(post_gamma)
    N, D = (dH if dY is None else dY).shape
    S, R = (CHAIN + 8) * U, (row_chain(N) + 8) * U
    out = {}
    dh, mag, dm = torch.zeros(N, D, dtype=torch.float64), torch.zeros(N, D, dtype=torch.float64), 0.0
    hh, r, m, direct = dh, 0.0, 0.0, dh
    if dH is not None:
        dh, mag, direct = dh + dH, mag + dH.abs(), direct + dH.abs()
    if dY is not None:
        r = _d(rstd)[:, None]
        t, hh = gamma * dY, H * r
        m, dm = (hh * t).mean(1, keepdim=True), S * (hh * t).abs().mean(1, keepdim=True)
        dh = dh + r * (t - hh * m)
        direct = direct + (r * t).abs()
        mag = mag + (r * t).abs() + (r * hh * m).abs()
        out["dgamma"] = ((dY * hh).sum(0), R * (dY * hh).abs().sum(0))
    ddh = 8 * U * mag + (r * hh * dm).abs()
    out["dR"] = (dh, ddh)
    g = 1.0 if gate is None else gate
    du = scale * g * dh
    ddu = (torch.as_tensor(scale * g, dtype=torch.float64).abs() * ddh) + 4 * U * du.abs()
    xh, u = X, X
    if post_gamma is not None:
        r1 = _d(post_rstd)[:, None]
        xh = X * r1
        u = xh * post_gamma

    def row_sum(w):  # sum of w dh as the kernels form it, and its bound
        e = (w * dh).sum(1, keepdim=True)
        spread = S * ((w.abs() * direct).sum(1, keepdim=True) + (r * m * (w * hh).abs().sum(1, keepdim=True) if dY is not None else 0.0) * torch.tensor(1.0).double()).abs()
        return e, spread + (abs(r) * dm * (w * hh).abs().sum(1, keepdim=True) if dY is not None else 0.0)

    if gate is not None:
        p = scale * dh * u
        dp = (scale * u).abs() * ddh + 6 * U * p.abs()
        if gate.dim() == 1:
            out["dgate"] = (p.sum(0), dp.sum(0) + R * p.abs().sum(0))
        elif gate.shape[1] == 1:
            e, de = row_sum(u)
            out["dgate"] = (scale * e, abs(scale) * de + 4 * U * (scale * e).abs())
        else:
            out["dgate"] = (p, dp)
    if post_gamma is None:
        out["dX"] = (du, ddu)
        return out
    w = u * (g if gate is None or gate.dim() == 1 or gate.shape[1] != 1 else 1.0)
    q = scale * (gate if gate is not None and gate.dim() == 2 and gate.shape[1] == 1 else 1.0)
    e, de = row_sum(w)
    m2, dm2 = q * e / D, torch.as_tensor(q, dtype=torch.float64).abs() * de / D + 4 * U * (q * e / D).abs()
    out["dX"] = (r1 * (post_gamma * du - xh * m2), (r1 * post_gamma).abs() * ddu + 6 * U * (r1 * post_gamma * du).abs() + (r1 * xh).abs() * dm2 + 6 * U * (r1 * xh * m2).abs())
    out["dpost_gamma"] = ((du * xh).sum(0), (ddu * xh.abs()).sum(0) + R * (du * xh).abs().sum(0))
    return out


def rotate(x, positions, turns, r, interleaved, factor=1.0, inverse=False):
    """(value, bound) of x [T, H, d] rotated; the angles from whole numbers: position times turns, modulo 2^64."""
    x = x.detach().cpu().double()
    angle = torch.tensor([[((int(p) * int(f)) % 2 ** 64) / 2.0 ** 64 * (2 * math.pi) for f in turns] for p in positions], dtype=torch.float64)
    co, si = (angle.cos() * factor)[:, None], (angle.sin() * factor * (-1.0 if inverse else 1.0))[:, None]
    out, tol = x.clone(), torch.zeros_like(x)
    if interleaved:
        ia, ib = torch.arange(0, r, 2), torch.arange(1, r, 2)
    else:
        ia, ib = torch.arange(r // 2), torch.arange(r // 2, r)
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * co - b * si, b * co + a * si
    # the angle within 2.4 roundings and 1.8e-9 of the polynomial, the polynomial's own, the products'
    tol[..., ia] = tol[..., ib] = (a.abs() + b.abs()) * abs(factor) * (8 * U + 4e-9)
    return out, tol


def slots(page_table, cache_lens, seq_starts, T, page_size, num_pages):
    """(slots, positions, bad): lists, and whether a page was missing."""
    at, pos, bad = [-1] * T, [0] * T, False
    for b in range(len(cache_lens)):
        for t in range(max(0, int(seq_starts[b])), min(T, int(seq_starts[b + 1]))):
            p = int(cache_lens[b]) + t - int(seq_starts[b])
            i = p // page_size
            page = int(page_table[b][i]) if cache_lens[b] >= 0 and i < page_table.shape[1] else -1
            if 0 <= page < num_pages:
                at[t], pos[t] = page * page_size + p % page_size, p
            else:
                bad = True
    return at, pos, bad
