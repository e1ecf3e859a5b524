"""Coefficients of the orthogonalisation whose small values shrink are refused: (0, 1, 0)
left nothing right after three rounds, its values far below what halves hold.  No GPU:
refused calls, and calls without matrices."""
import ctypes

import pytest

import sharded_optimizer_step_gb300 as ss
from sharded_optimizer_step_gb300 import _capi


@pytest.fixture(scope="module", autouse=True)
def _built():
    ss.build()


def _call(a, b, c, rounds):
    quintic = _capi.Quintic(a, b, c, 1e-7, rounds, 0)
    hp = (_capi.MuonHP * 1)(_capi.MuonHP(1e-3, 0.95, 0.1, 0.2, 1, 0))
    return (_capi.lib().matrices_orthogonalize(None, None, None, None, 0, 0, 0,
                                               ctypes.byref(quintic), None, 0, None),
            _capi.lib().tensors_muon_step(None, 0, 0, 0, hp, 1, ctypes.byref(quintic), None, None,
                                          None, 0, None))


@pytest.mark.parametrize("abc", [(0.0, 1.0, 0.0), (0.0, 0.0, 1.0), (0.999, -0.5, 0.0),
                                 (-0.5, 0.2, 0.0), (0.0, 0.0, 0.0)])
@pytest.mark.parametrize("rounds", [1, 3])
def test_shrinking_coefficients(abc, rounds):
    assert _call(*abc, rounds) == (_capi.ERR_INVALID, _capi.ERR_INVALID)
    assert b"shrink" in _capi.lib().shardstep_last_error()


@pytest.mark.parametrize("abc,rounds", [
    (ss.QUINTIC, 5), (ss.QUINTIC, 64), ((1.5, -0.5, 0.0), 24), ((1.875, -1.25, 0.375), 6),
    ((1.0, 0.0, 0.0), 3), ((1.0, -0.5, 0.0), 3), ((-1.0, 0.5, 0.0), 2)])
def test_taken_coefficients(abc, rounds):
    assert _call(*abc, rounds) == (_capi.OK, _capi.OK)
