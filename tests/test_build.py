"""What is built where (no GPU needed): libgma.so needs nvcc alone, its Python binding the installed torch."""
import os
import sys

import pytest

from linear_latent_routing_gb300 import build


@pytest.fixture(autouse=True)
def _built():
    build.build()


def test_library_alone_without_torch(monkeypatch, tmp_path):
    monkeypatch.setitem(sys.modules, "torch", None)            # as if it were not installed
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_block.so"))
    assert build.build() == build.LIB
    assert not os.path.exists(build.BINDING)


def test_binding_is_made_again_for_another_torch(monkeypatch, tmp_path):
    made = []
    monkeypatch.setattr(build, "_compile_binding", lambda *a: "object")
    monkeypatch.setattr(build, "_link_binding", lambda *a: made.append(a))
    build.build()
    assert not made
    other = tmp_path / "torch"
    (other / "lib").mkdir(parents=True)
    (other / "lib" / "libc10_cuda.so").write_text("")
    (other / "__init__.py").write_text("")
    (other / "version.py").write_text("__version__ = 'another'\n")
    monkeypatch.syspath_prepend(str(tmp_path))
    monkeypatch.delitem(sys.modules, "torch", raising=False)
    build.build()
    assert [a[-1] for a in made] == [str(other)]
    (other / "lib" / "libc10_cuda.so").unlink()                # a torch without CUDA: nothing to bind
    build.build()
    assert len(made) == 1
