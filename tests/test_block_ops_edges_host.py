"""Calls of the residual norms and of rotary positions at the edges of what is allowed, as far as the host decides
them.  No GPU: pointers are never dereferenced."""
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
