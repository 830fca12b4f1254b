"""What block_sparse_long_gb300.build takes for current, and what one part's failure leaves of the others."""
import os

import pytest

from block_sparse_long_gb300 import build as B


@pytest.fixture
def built(monkeypatch):
    B.build()
    assert B.up_to_date()


def test_another_torch_needs_another_module(built, monkeypatch):
    """The module is compiled against torch's headers; its file name does not tell which."""
    made = []
    monkeypatch.setattr(B, "_build_call", lambda: made.append(1))
    B.build()
    assert not made
    monkeypatch.setattr(B, "_torch_version", lambda: "__version__ = '0.0'")
    assert not B.up_to_date()
    B.build()
    assert made


def test_the_version_is_that_of_the_torch_that_is_imported():
    import torch
    assert f"'{torch.__version__}'" in B._torch_version()


def test_libraries_are_linked_whatever_becomes_of_the_module(monkeypatch, tmp_path):
    """A g++ that fails on the Python module is reported, and stops none of the CUDA libraries."""
    source, lib = tmp_path / "one.cu", str(tmp_path / "libone.so")
    source.write_text('extern "C" int one() { return 1; }\n')

    def fail():
        raise RuntimeError("g++ failed")
    for name, value in (("CSRC", str(tmp_path)), ("BUILD", str(tmp_path)), ("LIBRARIES", ((lib, ["one.cu"], [], []),)),
                        ("_call_stale", lambda: True), ("_build_call", fail)):
        monkeypatch.setattr(B, name, value)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        B.build()
    assert os.path.exists(lib)


def test_a_module_that_cannot_be_loaded_says_why(monkeypatch):
    from block_sparse_long_gb300 import attn

    def fail(*_):
        raise ImportError("undefined symbol: of another torch")
    monkeypatch.setattr(attn, "_module", None)
    monkeypatch.setattr(attn.importlib, "import_module", fail)
    with pytest.raises(RuntimeError, match="undefined symbol"):
        attn._calls()
