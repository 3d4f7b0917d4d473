"""The objectives' host side: what is refused and how the library is first loaded (no GPU)."""
import ctypes

import pytest

import convex_hull_pava_gb300 as chp
from convex_hull_pava_gb300 import objectives as obj


def test_temperature_whose_scale_leaves_float32():
    """log2(e) / T has to be a float32 number, not 1 / T alone."""
    lib = chp.load_library()
    p, ws = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x100000)
    for t in (3e-39, 4.2e-39):
        assert lib.iso_token_logp(p, 0, 4, 10, 10, p, t, p, p, ws, 0, None, None) == chp.ISO_ERR_INVALID_ARG
        assert lib.iso_token_logp_backward(p, 0, 4, 10, 10, p, t, p, p, 1.0, None, 0, p, 10,
                                           None) == chp.ISO_ERR_INVALID_ARG
        assert lib.iso_policy_loss(p, 0, 4, 10, 10, p, t, p, p, None, None, 0.2, 0.2, 0.0, 1.0, p, p, p, p, p, None, 10,
                                   ws, 1 << 20, None, None) == chp.ISO_ERR_INVALID_ARG


def test_setup_after_a_failed_load(monkeypatch):
    """A first call that could not load the library leaves nothing half set up: the next one tries again."""
    import torch
    for name in ("_abi", "_dtypes", "_raw_stream"):
        monkeypatch.setattr(obj, name, None)
    calls = []

    def load():
        calls.append(1)
        if len(calls) == 1:
            raise RuntimeError("no library yet")
        return chp.load_library()

    monkeypatch.setattr(obj, "load_library", load)
    x = torch.zeros(2, 4)
    with pytest.raises(RuntimeError):
        obj._scores(x)
    assert obj._dtypes is None   # what the calls look at
    with pytest.raises(ValueError):
        obj._scores(x)           # (a host tensor)
    assert len(calls) == 2 and obj._abi is not None and obj._raw_stream is not None
