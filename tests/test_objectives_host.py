"""The objectives' host side: what is refused and how the library is first loaded (no GPU)."""
import pytest

import convex_hull_pava_gb300 as chp
from convex_hull_pava_gb300 import objectives as obj


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
