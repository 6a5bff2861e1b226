"""Tests that call the library with addresses of nothing do not run where there is a GPU to read them."""
import importlib
from types import SimpleNamespace

import pytest

import conftest


@pytest.mark.parametrize("module,name", sorted(conftest.MADE_UP_ADDRESSES))
def test_skipped_where_a_gpu_is(monkeypatch, module, name):
    m = importlib.import_module(module)
    assert callable(getattr(m, name))
    item = SimpleNamespace(module=m, name=name + "[a]", originalname=name)
    monkeypatch.setattr(conftest, "gpu_is_here", lambda: True)
    with pytest.raises(pytest.skip.Exception):
        conftest.pytest_runtest_setup(item)
    conftest.pytest_runtest_setup(SimpleNamespace(module=m, name="test_sizes", originalname="test_sizes"))
    monkeypatch.setattr(conftest, "gpu_is_here", lambda: False)
    conftest.pytest_runtest_setup(item)
