"""The build of the library and of its tensor binding: the first does not depend on the second, and a binding made for another torch is
neither kept nor loaded."""
import os

import pytest

from fp8_causal_prefill_gb300 import ZyfaError, build, paged


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A build of one small source into a directory of its own."""
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libzyfa.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_paged.so"))
    monkeypatch.setattr(build, "SOURCES", ["zyfa_api.cu"])
    return tmp_path


def test_library_is_linked_where_the_binding_cannot_be_compiled(elsewhere, monkeypatch):
    def no_headers():
        raise RuntimeError("no torch headers here")

    monkeypatch.setattr(build, "compile_binding", no_headers)
    with pytest.raises(RuntimeError, match="no torch headers"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


def test_binding_of_another_torch_is_built_anew(elsewhere, monkeypatch):
    made = []

    def compiled():
        made.append(len(made))
        return "binding.o"

    def linked(obj):
        open(build.BINDING, "w").close()
        with open(os.path.join(build.BUILD, build.BINDING_STAMP), "w") as f:
            f.write(build._binding_target())

    monkeypatch.setattr(build, "compile_binding", compiled)
    monkeypatch.setattr(build, "link_binding", linked)
    build.build()
    build.build()
    assert made == [0]
    with open(os.path.join(build.BUILD, build.BINDING_STAMP), "w") as f:
        f.write("torch 1.0 python 3.0")
    build.build()
    build.build()
    assert made == [0, 1]


def test_binding_of_another_torch_is_not_loaded(elsewhere, monkeypatch):
    os.makedirs(build.BUILD)
    with open(os.path.join(build.BUILD, build.BINDING_STAMP), "w") as f:
        f.write("torch 1.0 python 3.0")
    monkeypatch.setattr(paged, "_native", None)
    with pytest.raises(ZyfaError, match="torch 1.0"):
        paged._load()


def test_build_leaves_a_stamp():
    build.build()
    assert build.binding_built_for() == build._binding_target()
