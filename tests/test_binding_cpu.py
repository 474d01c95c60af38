"""The Python binding without a GPU: what it imports, and the calls that it refuses before the library is reached."""
import builtins

import pytest
import torch

import token_level_sparse_gb300 as T


@pytest.fixture
def context(monkeypatch):
    """Contexts of no library: every call that passes the binding's checks is an error."""
    monkeypatch.setattr(T, "ts_create", lambda cfg: 1)
    monkeypatch.setattr(T, "ts_destroy", lambda handle: None)
    return T.Context


def test_a_context_needs_no_torch(context, monkeypatch):
    real = builtins.__import__

    def refuse(name, *a, **kw):
        if name == "torch" or name.startswith("torch."):
            raise ImportError(name)
        return real(name, *a, **kw)

    monkeypatch.setattr(builtins, "__import__", refuse)
    with pytest.raises(ImportError):
        import torch as _                                          # noqa: F401
    c = context(8, 2, 128, T.TS_KV_Q4, 2, 4, 8)
    assert c.max_tokens == 64
    c.close()
