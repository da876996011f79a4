"""The C library is built also where the torch binding cannot be (no torch headers,
no host compiler): the compile and link steps stood in for."""
import pytest

from fp8_dynamic_quantization_amd import build as b


@pytest.fixture
def linked(monkeypatch, tmp_path):
    out = []
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    monkeypatch.setattr(b, "_compile", lambda src: src)
    monkeypatch.setattr(b, "_link", lambda cmd, to: out.append((to, cmd)))
    return out


def test_library_without_the_binding(monkeypatch, linked):
    def no_headers():
        raise RuntimeError("compiling torch_binding.cpp failed")

    monkeypatch.setattr(b, "_compile_binding", no_headers)
    with pytest.raises(RuntimeError, match="torch_binding"):
        b.build()
    assert [to for to, _ in linked] == [b.LIB]
    assert set(b.SOURCES) <= set(linked[0][1])


def test_binding_is_linked_after_the_library(monkeypatch, linked):
    monkeypatch.setattr(b, "_compile_binding", lambda: "binding.o")
    assert b.build() == b.LIB
    assert [to for to, _ in linked] == [b.LIB, b.BINDING]
    assert "binding.o" in linked[1][1]
