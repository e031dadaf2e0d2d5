"""What the residual norms, rotary positions and the paged cache refuse before anything is enqueued, the
rotary frequencies, and the 64-bit references themselves.  No GPU: pointers are never dereferenced."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

import block_ops_ref as ref

P = 0x10000  # aligned fake device addresses
Q = 0x20000


@pytest.fixture(scope="module")
def so():
    import __graft_entry__

    __graft_entry__._build_module().build()
    import cross_entropy_loss_gb300 as ce

    return ce


# ------------------------------------------------------------------- residual norms
FWD = dict(X=P, ldx=64, R=P, ldr=64, dtype=1, N=4, D=64, gate=None, kind=0, ldg=0, post_gamma=None, gamma=P, scale=1.0, post_eps=1e-5, eps=1e-5, H=P, ldh=64, Y=Q, ldy=64, post_rstd=None, rstd=P, stream=None)
BWD = dict(dY=P, lddy=64, dH=P, lddh=64, H=P, ldh=64, X=P, ldx=64, dtype=1, N=4, D=64, gate=None, kind=0, ldg=0, post_gamma=None, gamma=P, post_rstd=None, rstd=P, scale=1.0, dR=P, lddr=64, dX=Q, lddx=64, dgamma=P, dgate=None, lddg=0, dpost_gamma=None, ws=P, wsb=1 << 24, stream=None)


def _call(so, fn, base, **change):
    assert not set(change) - set(base)
    so.lib.foak_test_fail_next_launches(1)  # a call that is not refused ends here
    try:
        return getattr(so.lib, fn)(*{**base, **change}.values())
    finally:
        so.lib.foak_test_fail_next_launches(0)


@pytest.mark.parametrize("change,status", [
    ({}, "CUDA"), ({"dtype": 2}, "UNSUPPORTED"), ({"D": 60}, "UNSUPPORTED"), ({"D": 32776, "ldx": 1 << 16}, "UNSUPPORTED"),
    ({"D": 0}, "INVALID_ARG"), ({"N": -1}, "INVALID_ARG"), ({"ldx": 56}, "INVALID_ARG"), ({"ldr": 56}, "INVALID_ARG"),
    ({"ldh": 56}, "INVALID_ARG"), ({"ldy": 56}, "INVALID_ARG"), ({"ldx": 68}, "INVALID_ARG"), ({"X": P + 2}, "INVALID_ARG"),
    ({"X": None}, "INVALID_ARG"), ({"R": None}, "INVALID_ARG"), ({"H": None}, "INVALID_ARG"), ({"Y": None}, "INVALID_ARG"),
    ({"Y": P}, "INVALID_ARG"), ({"gamma": None}, "INVALID_ARG"), ({"gamma": None, "Y": None}, "INVALID_ARG"),
    ({"gamma": None, "Y": None, "rstd": None}, "CUDA"), ({"gamma": P + 8}, "INVALID_ARG"), ({"post_gamma": P + 8}, "INVALID_ARG"),
    ({"post_gamma": P, "post_rstd": P}, "CUDA"), ({"post_rstd": P}, "INVALID_ARG"), ({"rstd": P + 2}, "INVALID_ARG"),
    ({"scale": math.nan}, "INVALID_ARG"), ({"scale": math.inf}, "INVALID_ARG"), ({"eps": -1e-9}, "INVALID_ARG"),
    ({"eps": math.nan}, "INVALID_ARG"), ({"post_eps": -1.0}, "INVALID_ARG"), ({"kind": 4}, "INVALID_ARG"), ({"kind": -1}, "INVALID_ARG"),
    ({"kind": 1}, "INVALID_ARG"), ({"gate": P}, "INVALID_ARG"), ({"gate": P, "kind": 1}, "CUDA"), ({"gate": P + 2, "kind": 1}, "INVALID_ARG"),
    ({"gate": P + 2, "kind": 2, "ldg": 1}, "CUDA"), ({"gate": P + 1, "kind": 2, "ldg": 1}, "INVALID_ARG"), ({"gate": P, "kind": 2}, "INVALID_ARG"),
    ({"gate": P, "kind": 3, "ldg": 64}, "CUDA"), ({"gate": P, "kind": 3, "ldg": 56}, "INVALID_ARG"), ({"gate": P + 2, "kind": 3, "ldg": 64}, "INVALID_ARG"),
    ({"ldh": 72}, "INVALID_ARG"), ({"ldh": 72, "N": 1}, "CUDA"), ({"ldx": 72, "ldr": 72, "ldh": 72}, "CUDA"),
    ({"N": 0, "X": None, "R": None, "H": None, "Y": None}, "CUDA")])
def test_forward_refusals(so, change, status):
    assert _call(so, "foak_residual_norm_forward", FWD, **change) == getattr(so, "FOAK_ERR_" + status)


@pytest.mark.parametrize("change,status", [
    ({}, "CUDA"), ({"dtype": 9}, "UNSUPPORTED"), ({"D": 12}, "UNSUPPORTED"), ({"N": -2}, "INVALID_ARG"), ({"dY": None, "dH": None}, "INVALID_ARG"),
    ({"dY": None}, "INVALID_ARG"), ({"dY": None, "dgamma": None}, "CUDA"), ({"dY": None, "dgamma": None, "H": None, "gamma": None, "rstd": None}, "CUDA"),
    ({"dH": None}, "CUDA"), ({"H": None}, "INVALID_ARG"), ({"rstd": None}, "INVALID_ARG"), ({"gamma": None}, "INVALID_ARG"), ({"dR": None}, "INVALID_ARG"),
    ({"dX": None}, "CUDA"), ({"dX": P}, "INVALID_ARG"), ({"X": None}, "CUDA"), ({"post_gamma": P, "post_rstd": P, "X": None}, "INVALID_ARG"),
    ({"post_gamma": P}, "INVALID_ARG"), ({"post_gamma": P, "post_rstd": P, "dpost_gamma": P}, "CUDA"), ({"dpost_gamma": P}, "INVALID_ARG"),
    ({"dgate": P}, "INVALID_ARG"), ({"gate": P, "kind": 1, "dgate": P}, "CUDA"), ({"gate": P, "kind": 1, "dgate": P, "X": None}, "INVALID_ARG"),
    ({"gate": P, "kind": 3, "ldg": 64, "dgate": 0x30000, "lddg": 64}, "CUDA"), ({"gate": P, "kind": 3, "ldg": 64, "dgate": 0x30000, "lddg": 56}, "INVALID_ARG"),
    ({"gate": P, "kind": 3, "ldg": 64, "dgate": P, "lddg": 64}, "INVALID_ARG"), ({"gate": P, "kind": 3, "ldg": 64, "dgate": Q, "lddg": 64}, "INVALID_ARG"),
    ({"lddr": 72}, "INVALID_ARG"), ({"lddy": 8}, "INVALID_ARG"), ({"lddh": 8}, "INVALID_ARG"), ({"ldh": 8}, "INVALID_ARG"), ({"lddx": 8}, "INVALID_ARG"),
    ({"scale": math.nan}, "INVALID_ARG"), ({"dgamma": P + 2}, "INVALID_ARG"), ({"ws": None}, "WORKSPACE"), ({"ws": P + 16}, "WORKSPACE"),
    ({"wsb": 1000}, "WORKSPACE"), ({"N": 0, "dY": None, "dH": None, "dR": None, "dX": None, "X": None}, "CUDA")])
def test_backward_refusals(so, change, status):
    assert _call(so, "foak_residual_norm_backward", BWD, **change) == getattr(so, "FOAK_ERR_" + status)


def test_workspace_size(so):
    assert so.foak_residual_norm_workspace_size(-1, 64) == 0 and so.foak_residual_norm_workspace_size(4, 40000) == 0
    assert so.foak_residual_norm_workspace_size(8192, 4096) >= 2 * 128 * 4096 * 4


# ----------------------------------------------------------- rotary positions, paged cache
ROT = dict(Q=P, ldq=256, ldqh=64, Qo=Q, ldqo=256, ldqoh=64, Hq=4, K=P, ldk=128, ldkh=64, Ko=Q, ldko=128, ldkoh=64, Hk=2, dtype=1, T=3, d=64, r=64, interleaved=0, positions=P, turns=P, factor=1.0, inverse=0, stream=None)
SLOTS = dict(table=P, ld=4, most=4, lens=P, starts=P, B=2, T=3, page=16, pages=8, slots=P, positions=P, err=P, stream=None)
APP = dict(K=P, ldk=128, ldkh=64, V=P, ldv=128, ldvh=64, Hk=2, dtype=1, T=3, d=64, dv=64, slots=P, kc=P, kp=2048, kpl=128, kh=64, vc=Q, vp=2048, vpl=128, vh=64, pages=8, page=16, Q=P, ldq=256, ldqh=64, Qo=Q, ldqo=256, ldqoh=64, Hq=4, r=64, interleaved=0, positions=P, turns=P, factor=1.0, err=None, stream=None)


@pytest.mark.parametrize("change,status", [
    ({}, "CUDA"), ({"dtype": 5}, "UNSUPPORTED"), ({"r": 0}, "UNSUPPORTED"), ({"r": 63}, "UNSUPPORTED"), ({"r": 66}, "UNSUPPORTED"), ({"T": -1}, "INVALID_ARG"),
    ({"Q": None}, "CUDA"), ({"K": None}, "CUDA"), ({"Qo": None}, "INVALID_ARG"), ({"Q": P + 1}, "INVALID_ARG"), ({"Q": P + 2}, "CUDA"), ({"ldq": -256}, "INVALID_ARG"),
    ({"ldqoh": 32}, "INVALID_ARG"), ({"ldqo": 0}, "INVALID_ARG"), ({"Hq": -1}, "INVALID_ARG"), ({"Hq": 1 << 24}, "INVALID_ARG"), ({"positions": None}, "INVALID_ARG"),
    ({"positions": P + 4}, "INVALID_ARG"), ({"turns": None}, "INVALID_ARG"), ({"turns": P + 4}, "INVALID_ARG"), ({"factor": math.nan}, "INVALID_ARG"),
    ({"Qo": P}, "CUDA"), ({"Qo": P, "ldqo": 320}, "INVALID_ARG"), ({"Qo": P, "ldqoh": 72}, "INVALID_ARG"), ({"T": 0, "Q": None, "K": None, "turns": None}, "CUDA")])
def test_rotary_refusals(so, change, status):
    assert _call(so, "foak_rotary_apply", ROT, **change) == getattr(so, "FOAK_ERR_" + status)


@pytest.mark.parametrize("change,status", [
    ({}, "CUDA"), ({"page": 0}, "INVALID_ARG"), ({"pages": 0}, "INVALID_ARG"), ({"T": -1}, "INVALID_ARG"), ({"B": -1}, "INVALID_ARG"), ({"ld": 3}, "INVALID_ARG"),
    ({"table": None}, "INVALID_ARG"), ({"lens": None}, "INVALID_ARG"), ({"starts": None}, "INVALID_ARG"), ({"slots": None}, "INVALID_ARG"), ({"positions": P + 4}, "INVALID_ARG"),
    ({"err": P + 2}, "INVALID_ARG"), ({"pages": 1 << 40, "page": 1 << 30}, "UNSUPPORTED"), ({"T": 1 << 31}, "UNSUPPORTED"), ({"B": 0, "table": None, "lens": None}, "CUDA")])
def test_slots_refusals(so, change, status):
    assert _call(so, "foak_kv_slots", SLOTS, **change) == getattr(so, "FOAK_ERR_" + status)


@pytest.mark.parametrize("change,status", [
    ({}, "CUDA"), ({"dtype": 2}, "UNSUPPORTED"), ({"r": 30000}, "UNSUPPORTED"), ({"r": 0}, "INVALID_ARG"), ({"r": 0, "Q": None, "turns": None, "positions": None}, "CUDA"),
    ({"Q": None}, "CUDA"), ({"K": None}, "INVALID_ARG"), ({"V": None}, "INVALID_ARG"), ({"kc": None}, "INVALID_ARG"), ({"vc": P}, "INVALID_ARG"), ({"Hk": 0}, "INVALID_ARG"),
    ({"slots": None}, "INVALID_ARG"), ({"slots": P + 4}, "INVALID_ARG"), ({"kp": 0}, "INVALID_ARG"), ({"vpl": 0}, "INVALID_ARG"), ({"kh": 32}, "INVALID_ARG"), ({"vh": 32}, "INVALID_ARG"),
    ({"page": 0}, "INVALID_ARG"), ({"pages": 0}, "INVALID_ARG"), ({"pages": 1 << 60}, "UNSUPPORTED"), ({"dv": 0}, "INVALID_ARG"), ({"positions": None}, "INVALID_ARG"),
    ({"turns": None}, "INVALID_ARG"), ({"Qo": None}, "INVALID_ARG"), ({"Qo": P, "ldqo": 512}, "INVALID_ARG"), ({"err": P + 1}, "INVALID_ARG"), ({"factor": math.inf}, "INVALID_ARG"),
    ({"T": 0, "K": None, "V": None, "slots": None}, "CUDA")])
def test_append_refusals(so, change, status):
    assert _call(so, "foak_kv_append", APP, **change) == getattr(so, "FOAK_ERR_" + status)


def test_status_of_a_page(so):
    assert so.status_string(so.FOAK_ERR_PAGE_RANGE).startswith("FOAK_ERR_PAGE_RANGE")


# ---------------------------------------------------------------------- frequencies
def test_frequencies(so):
    """Formulas written out again; numbers of a 64-bit power and a few products: 1e-13 relative."""
    r, base, factor, low, high, original = 128, 500000.0, 8.0, 1.0, 4.0, 8192.0
    plain = [base ** (-2.0 * i / r) for i in range(r // 2)]

    def close(got, want):
        assert len(got) == len(want) and all(abs(a - b) <= 1e-13 * b for a, b in zip(got, want))

    close(so.foak_rotary_inv_freq(r, base=base), plain)
    close(so.foak_rotary_inv_freq(r, base=base, scaling="linear", factor=factor), [f / factor for f in plain])
    wide = base * factor ** (r / (r - 2))
    close(so.foak_rotary_inv_freq(r, base=base, scaling="ntk", factor=factor), [wide ** (-2.0 * i / r) for i in range(r // 2)])
    bands = []
    for f in plain:
        n = original * f / (2 * math.pi)
        w = min(1.0, max(0.0, (n - low) / (high - low)))
        bands.append(w * f + (1 - w) * f / factor)
    got = so.foak_rotary_inv_freq(r, base=base, scaling="bands", factor=factor, low=low, high=high, original=original)
    assert all(abs(a - b) <= 1e-12 * b for a, b in zip(got, bands))
    assert got[0] == plain[0] and abs(got[-1] * factor / plain[-1] - 1) < 1e-13
    first = math.floor(r * math.log(original / (32.0 * 2 * math.pi)) / (2 * math.log(base)))
    last = math.ceil(r * math.log(original / (1.0 * 2 * math.pi)) / (2 * math.log(base)))
    ramp = [f * (1 - w) + f / factor * w for i, f in enumerate(plain) for w in [min(1.0, max(0.0, (i - first) / (last - first)))]]
    close(so.foak_rotary_inv_freq(r, base=base, scaling="ramp", factor=factor, original=original), ramp)
    # one frequency alone, and a context shorter than a turn: finite
    assert all(math.isfinite(f) for f in so.foak_rotary_inv_freq(2, scaling="ramp", factor=2.0, original=1.0))


def test_turns(so):
    """Within 2^-53 of the turns a position, relatively: the division's and the constant's roundings."""
    pi = Fraction("3.14159265358979323846264338327950288419716939937510")
    freqs = [1.0, 0.5, 1e-3, 3.7e-7, 6.0, 100.0, -0.25, 0.0, 2 * math.pi]
    for f, t in zip(freqs, so.foak_rotary_turns(freqs).tolist()):
        want = Fraction(f) / (2 * pi)
        off = (Fraction(t % 2 ** 64, 2 ** 64) - want) % 1
        off = min(off, 1 - off)
        assert off <= abs(want) * Fraction(1, 2 ** 52) + Fraction(1, 2 ** 53), f


def test_frequency_refusals(so):
    out = (ctypes.c_double * 64)()
    call = lambda *a: so.lib.foak_rotary_inv_freq(*a, out)  # noqa: E731
    assert call(1e4, 64, 0, 1.0, 1.0, 4.0, 0.0) == so.FOAK_OK
    for args in ((1.0, 64, 0, 1.0, 1.0, 4.0, 0.0), (math.inf, 64, 0, 1.0, 1.0, 4.0, 0.0), (1e4, 64, 5, 2.0, 1.0, 4.0, 8.0), (1e4, 64, 1, 0.5, 1.0, 4.0, 8.0),
                 (1e4, 64, 3, 2.0, 4.0, 1.0, 8.0), (1e4, 64, 3, 2.0, 1.0, 4.0, 0.0), (1e4, 64, 4, 2.0, 0.0, 4.0, 8.0), (1e4, 64, 4, math.nan, 1.0, 4.0, 8.0)):
        assert call(*args) == so.FOAK_ERR_INVALID_ARG, args
    assert call(1e4, 63, 0, 1.0, 1.0, 4.0, 0.0) == so.FOAK_ERR_UNSUPPORTED and call(1e4, 2, 2, 2.0, 1.0, 4.0, 0.0) == so.FOAK_ERR_UNSUPPORTED
    with pytest.raises(so.FoakError):
        so.foak_rotary_turns([1.0, math.nan])
    for bad in (lambda: so.foak_rotary_plan(64, scaling="wide", device="cpu"), lambda: so.foak_rotary_plan(63, device="cpu"),
                lambda: so.foak_rotary_plan(64, inv_freq=[1.0], device="cpu"), lambda: so.foak_rotary_plan(64, attention_factor=math.nan, device="cpu")):
        with pytest.raises(ValueError):
            bad()


# --------------------------------------------------------------- the references themselves
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "row", "full"])
def test_reference_gradients(gate, post):
    """The backward formulas against automatic differentiation of the forward, both in 64 bits."""
    c = {k: None if v is None else v.double() for k, v in ref.make_norm(5, 24, "f32", gate, post, seed=4).items()}
    names = [k for k in ("X", "R", "gamma", "gate", "post_gamma") if c[k] is not None]
    for k in names:
        c[k].requires_grad_(True)
    u = c["X"]
    post_rstd = (u.square().mean(1) + 1e-6).rsqrt() if post else None
    if post:
        u = u * post_rstd[:, None] * c["post_gamma"]
    H = c["R"] + 0.22 * u * (1.0 if gate == "none" else c["gate"])
    rstd = (H.square().mean(1) + 1e-5).rsqrt()
    ((H * rstd[:, None] * c["gamma"] * c["dY"]).sum() + (H * c["dH"]).sum()).backward()
    f = ref.norm_forward(c["X"], c["R"], c["gamma"], c["gate"], c["post_gamma"], 0.22, 1e-5, 1e-6)
    torch.testing.assert_close(f["H"][0], H.detach(), rtol=1e-12, atol=1e-12)
    want = ref.norm_backward(c["dY"], c["dH"], H, rstd, c["gamma"], c["X"], c["gate"], c["post_gamma"], post_rstd, 0.22)
    assert sorted(want) == sorted("d" + k for k in names)
    for k in names:
        torch.testing.assert_close(want["d" + k][0], c[k].grad.reshape(want["d" + k][0].shape), rtol=1e-10, atol=1e-11)


def test_a_wrong_result_is_noticed():
    x = torch.randn(4, 2, 8)
    turns = [2 ** 60, 2 ** 59]
    good, tol = ref.rotate(x, [1, 2, 3, 4], turns, 4, False)
    ref.assert_close(good.float(), (good, tol), "as it is")
    for wrong in (ref.rotate(x, [1, 2, 3, 5], turns, 4, False)[0], ref.rotate(x, [1, 2, 3, 4], turns, 4, True)[0], ref.rotate(x, [1, 2, 3, 4], turns, 4, False, inverse=True)[0]):
        with pytest.raises(AssertionError):
            ref.assert_close(wrong.float(), (good, tol), "another")
