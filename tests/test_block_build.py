"""The library is built where the compiled argument checks cannot be: without a host compiler, or without its headers."""
import warnings

import pytest

from all_reduce_reduction_ring_amd import build as b


@pytest.fixture
def away(monkeypatch, tmp_path):
    """A build into tmp_path that compiles no HIP source."""
    linked = []
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "objs"))
    for name in ("LIB", "CEILING_LIB", "MARSHAL_LIB"):
        monkeypatch.setattr(b, name, str(tmp_path / name))
    monkeypatch.setattr(b, "_compile", lambda unit: "".join([unit[0], *unit[1]]))
    monkeypatch.setattr(b, "_link", lambda objs, out: linked.append(out))
    (tmp_path / "MARSHAL_LIB").write_text("of an older build")
    return tmp_path, linked


@pytest.mark.parametrize("compiler", ["/nowhere/g++", "false"])
def test_no_host_compiler(away, monkeypatch, compiler):
    tmp_path, linked = away
    monkeypatch.setattr(b, "CXX", compiler)
    with pytest.warns(UserWarning, match="_marshal.so was not built"):
        assert b.build(jobs=1) == b.LIB
    assert linked == [b.LIB, b.CEILING_LIB] and not (tmp_path / "MARSHAL_LIB").exists()


def test_no_torch(away, monkeypatch):
    monkeypatch.setitem(__import__("sys").modules, "torch", None)
    with pytest.warns(UserWarning, match="_marshal.so was not built"):
        assert b.build(jobs=1) == b.LIB


def test_a_whole_build(away):
    tmp_path, linked = away
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        b.build(jobs=1)
    assert (tmp_path / "MARSHAL_LIB").stat().st_size > 10_000 and len(linked) == 2


def test_a_source_that_does_not_compile_still_ends_the_build(away, monkeypatch):
    def fail(unit):
        raise RuntimeError("hipcc failed")

    monkeypatch.setattr(b, "_compile", fail)
    with pytest.raises(RuntimeError, match="hipcc failed"):
        b.build(jobs=1)
