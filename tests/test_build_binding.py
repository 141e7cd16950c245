"""The native binding of the tree-decoding calls and the library are built apart:
where the binding cannot be built, the rest of the library can (no GPU needed)."""

import os

import pytest


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build with a binding of its own, to be made anew."""
    from self_speculative_decoding_gb300 import build as b
    b.build()
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(b, "STAMP", str(tmp_path / "_binding.txt"), raising=False)
    return b


def test_the_library_is_built_without_pytorchs_headers(build, monkeypatch, tmp_path):
    import torch

    import self_speculative_decoding_gb300 as ssd
    assert build.binding_failure() == "it has not been built"
    with monkeypatch.context() as m:
        m.setattr(torch, "__file__", str(tmp_path / "torch" / "__init__.py"))
        before = os.path.getmtime(build.LIB)
        with pytest.warns(UserWarning, match="tree-decoding calls"):
            assert build.build() == build.LIB
        assert os.path.getmtime(build.LIB) == before and not os.path.exists(build.BINDING)
        # the calls say why, and the attempt is not made again until something changes
        m.setattr(ssd, "_native", None)
        with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
            ssd.ops.beam_select(None, None, 1)
        m.setattr(build, "_compile_binding", lambda: pytest.fail("tried again"))
        assert build.build() == build.LIB


def test_a_binding_of_another_pytorch_is_built_anew(build, monkeypatch):
    import self_speculative_decoding_gb300 as ssd
    made = []
    monkeypatch.setattr(build, "_compile_binding", lambda: made.append(open(build.BINDING, "w").close()))
    build.build()
    build.build()
    assert len(made) == 1 and build.binding_failure() == ""
    text = open(build.STAMP).read()
    with open(build.STAMP, "w") as f:
        f.write(text.replace("PyTorch ", "PyTorch 0."))
    assert "built against PyTorch 0." in build.binding_failure()
    monkeypatch.setattr(ssd, "_native", None)
    with pytest.raises(RuntimeError, match="built against"):
        ssd.ops.beam_select(None, None, 1)
    build.build()
    assert len(made) == 2 and build.binding_failure() == ""
    os.remove(build.BINDING)
    build.build()
    assert len(made) == 3


def test_a_binding_that_fails_takes_an_old_one_along(build, monkeypatch):
    open(build.BINDING, "w").close()

    def fail():
        raise RuntimeError("no compiler")

    monkeypatch.setattr(build, "_compile_binding", fail)
    with pytest.warns(UserWarning, match="no compiler"):
        build.build()
    assert not os.path.exists(build.BINDING) and build.binding_failure() == "no compiler"


def test_a_binding_that_does_not_load_is_named(monkeypatch):
    import sys

    import self_speculative_decoding_gb300 as ssd
    monkeypatch.setattr(ssd, "_native", None)
    monkeypatch.delattr(ssd, "_binding", raising=False)
    monkeypatch.setitem(sys.modules, ssd.__name__ + "._binding", None)
    with pytest.raises(RuntimeError, match="native binding"):
        ssd.ops.beam_select(None, None, 1)
