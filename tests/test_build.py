"""The build: the library without torch or a working front end, and _front's torch."""
import os

import pytest

from all_gather_gemm_chunked_gb300 import build as b


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A library of one function, in a folder of its own."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(b, "sources", lambda: [str(src)])
    for name, file in (("LIB", "libone.so"), ("FRONT", "_front.so"), ("BUILD_DIR", "build")):
        monkeypatch.setattr(b, name, str(tmp_path / file))
    return tmp_path


def test_library_without_torch(small, monkeypatch):
    monkeypatch.setattr(b, "_has_torch", lambda: False)
    assert not b.up_to_date()
    assert b.build() == b.LIB and os.path.exists(b.LIB) and not os.path.exists(b.FRONT)
    assert b.up_to_date()


def test_library_is_there_where_the_front_end_fails(small, monkeypatch):
    def fails(verbose=False):
        raise RuntimeError("g++ failed")

    monkeypatch.setattr(b, "_has_torch", lambda: True)
    monkeypatch.setattr(b, "_compile_front", fails)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        b.build()
    assert os.path.exists(b.LIB) and b.library_up_to_date() and not b.up_to_date()


def test_front_belongs_to_one_torch(monkeypatch):
    torch = pytest.importorskip("torch")
    b.build()
    assert b.up_to_date() and b.front_up_to_date()
    monkeypatch.setattr(torch, "__version__", "1.2.3+other")
    assert not b.front_up_to_date() and not b.up_to_date() and b.library_up_to_date()


def test_a_front_of_another_torch_is_refused():
    pytest.importorskip("torch")
    b.build()
    from all_gather_gemm_chunked_gb300 import moe
    assert moe._same_torch("2.9.1", "2.9.1") and moe._same_torch("2.11.0", "2.11.0+cu130")
    assert moe._same_torch("2.9.1", "2.9.1a0+git12") and not moe._same_torch("2.9.1", "2.11.0+cu130")
    assert not moe._same_torch("2.1.0", "2.1.01")
