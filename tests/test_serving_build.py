"""The serving step's compiled binding belongs to the torch and Python that it was built against."""
import sysconfig

import pytest
import torch

from quantized_int8_gemm_gb300 import build, serving


@pytest.fixture
def built():
    build.build()
    assert build.up_to_date()


def test_a_binding_of_another_torch_is_not_used(built, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    assert not build.up_to_date()
    monkeypatch.setattr(serving, "_binding", None)
    with pytest.raises(RuntimeError, match="not built"):
        serving._load()


def test_a_binding_of_another_python_is_not_used(built, monkeypatch):
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399" if name == "SOABI" else real(name))
    assert not build.up_to_date()
    monkeypatch.setattr(serving, "_binding", None)
    with pytest.raises(RuntimeError, match="not built"):
        serving._load()


def test_the_built_binding_loads(built, monkeypatch):
    monkeypatch.setattr(serving, "_binding", None)
    assert serving._load() is serving._binding and hasattr(serving._binding, "paged_attention")
