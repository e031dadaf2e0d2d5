"""Calls of the residual norms and of rotary positions at the edges of what is allowed, as far as the host decides
them.  No GPU: pointers are never dereferenced."""
import math
from fractions import Fraction

import pytest

from test_block_ops_host import BWD, FWD, P, _call, so  # noqa: F401  (the library, a fixture)


@pytest.mark.parametrize("change,status", [
    ({"kind": 1}, "INVALID_ARG"), ({"kind": 1, "gate": P}, "CUDA"), ({"kind": 2, "ldg": 1}, "CUDA"), ({"kind": 3, "ldg": 64}, "CUDA"), ({"gate": P}, "INVALID_ARG")])
def test_gate_of_an_empty_batch(so, change, status):  # noqa: F811
    """A gate a channel has D values however many rows there are; one a row or an element has none of no rows."""
    none = {"N": 0, "X": None, "R": None, "H": None, "Y": None}
    assert _call(so, "foak_residual_norm_forward", FWD, **none, **change) == getattr(so, "FOAK_ERR_" + status)
    none = {"N": 0, "dY": None, "dH": None, "H": None, "X": None, "rstd": None, "dR": None, "dX": None}
    assert _call(so, "foak_residual_norm_backward", BWD, **none, **change) == getattr(so, "FOAK_ERR_" + status)


def test_gamma_of_an_empty_batch(so):  # noqa: F811
    """A gradient of Y needs the norm's weight, whose gradient goes over it, however many rows there are."""
    none = {"N": 0, "dH": None, "H": None, "X": None, "rstd": None, "dR": None, "dX": None}
    assert _call(so, "foak_residual_norm_backward", BWD, **none, dY=P, gamma=None) == so.FOAK_ERR_INVALID_ARG
    assert _call(so, "foak_residual_norm_backward", BWD, **none, dY=P, gamma=None, dgamma=None) == so.FOAK_ERR_INVALID_ARG
    assert _call(so, "foak_residual_norm_backward", BWD, **none, dY=P) == so.FOAK_ERR_CUDA
    assert _call(so, "foak_residual_norm_backward", BWD, **none, dY=None, gamma=None) == so.FOAK_ERR_CUDA


def test_turns_to_the_last_bit_but_one(so):  # noqa: F811
    """Each of the two parts that a fraction is made of is cut off below 2^-64 of a turn, and neither the constant's
    106 bits nor the second part's roundings add a hundredth of that below 2^40: less than 2^-63 in all."""
    pi = Fraction("3.141592653589793238462643383279502884197169399375105820974944592307816406286")
    freqs = [1.0, 0.5, -0.25, 1e-3, 3.7e-7, 1.9e-8, 6.0, 100.0, -100.0, 12345.678, 2.0 ** 39 + 0.1, 0.0, -1e-30, 5e-324, 2 * math.pi, 8 * math.pi]
    freqs += so.foak_rotary_inv_freq(128, base=500000.0) + so.foak_rotary_inv_freq(96, base=1e7, scaling="linear", factor=32.0)
    for f, t in zip(freqs, so.foak_rotary_turns(freqs).tolist()):
        off = (Fraction(t, 2 ** 64) - Fraction(f) / (2 * pi)) % 1
        assert min(off, 1 - off) <= Fraction(1, 2 ** 63), f
    assert len(so.foak_rotary_turns([1e300, -1e300, 1.7976931348623157e308])) == 3  # any number of turns is taken


def test_workspace_goes_by_the_rows(so):  # noqa: F811
    """Partial sums of as many groups as there can be, two of D floats each, and two floats a row; up to 255 bytes of
    rounding.  Of few rows little, of more rows no less."""
    size = so.foak_residual_norm_workspace_size
    for D in (8, 4096, 16384, 32768):
        assert 0 < size(0, D) <= size(1, D) <= 2 * D * 4 + 8 + 255
        assert size(100, D) <= 100 * (2 * D * 4 + 8) + 255
        sizes = [size(N, D) for N in (0, 1, 2, 127, 128, 129, 2431, 2432, 2433, 100000, 100001)]
        assert sizes == sorted(sizes)
        assert size(100001, D) >= 2 * 128 * D * 4
        change = {k: 1 << 16 for k in ("ldx", "lddy", "lddh", "ldh", "lddr", "lddx")}
        for N in (1, 100, 100001):
            assert _call(so, "foak_residual_norm_backward", BWD, N=N, D=D, wsb=size(N, D), **change) == so.FOAK_ERR_CUDA
            assert _call(so, "foak_residual_norm_backward", BWD, N=N, D=D, wsb=size(N, D) - 1, **change) == so.FOAK_ERR_WORKSPACE
