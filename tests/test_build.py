"""What building the library and the binding's C++ part needs, with stand-ins for the compilers."""
import os
import sys
import warnings

import pytest
import torch

import paged_kv_prep_gb300 as pkv
from paged_kv_prep_gb300 import _lib
from paged_kv_prep_gb300 import build as pbuild

COMPILER = """#!{python}
import sys
if {fails}:
    sys.exit("no such header")
open(sys.argv[sys.argv.index("-o") + 1], "w").close()
"""


@pytest.fixture
def places(tmp_path, monkeypatch):
    """A build into a folder of its own: a function that makes the compilers (nvcc, g++)."""
    for name in ("BUILD", "LIBRARY", "MARSHAL", "MARSHAL_ABI"):
        monkeypatch.setattr(pbuild, name, str(tmp_path / name.lower()))

    def compilers(fails=False, missing=False):
        for name, fail in (("NVCC", False), ("CXX", fails)):
            path = tmp_path / name
            path.write_text(COMPILER.format(python=sys.executable, fails=fail))
            path.chmod(0o755)
            monkeypatch.setenv(name, str(path if not (missing and name == "CXX") else tmp_path / "nowhere"))
    compilers()
    return compilers


def test_both_are_built(places):
    assert not pbuild.up_to_date()
    assert pbuild.build() == pbuild.LIBRARY
    assert os.path.exists(pbuild.LIBRARY) and os.path.exists(pbuild.MARSHAL) and pbuild.up_to_date()
    os.remove(pbuild.MARSHAL)
    assert not pbuild.up_to_date()


@pytest.mark.parametrize("what", ["torch", "Python", "unknown"])
def test_the_bindings_part_is_built_again_for_another_torch_or_python(places, monkeypatch, what):
    pbuild.build()
    assert pbuild.up_to_date() and pbuild.marshal_abi() == pbuild.abi(torch.__version__)
    if what == "torch":
        monkeypatch.setattr(pbuild, "_torch_version", lambda path: "2.0.0")
    elif what == "Python":
        monkeypatch.setattr(pbuild.sysconfig, "get_config_var", lambda name: "cpython-399")
    else:
        os.remove(pbuild.MARSHAL_ABI)
    assert not pbuild.up_to_date()
    pbuild.build()
    assert pbuild.up_to_date()


def test_the_bindings_part_of_another_torch_is_not_imported(places, monkeypatch):
    monkeypatch.setattr(_lib, "_SHORT", None)
    pbuild.build()
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    with pytest.warns(RuntimeWarning, match="for another torch or Python.*not for torch .*other"):
        assert _lib._short() is _lib._NoShort


def test_the_library_needs_no_torch(places, monkeypatch):
    found = pbuild.importlib.util.find_spec
    monkeypatch.setattr(pbuild.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else found(name, *a))
    places(missing=True)
    assert pbuild.build() == pbuild.LIBRARY
    assert os.path.exists(pbuild.LIBRARY) and not os.path.exists(pbuild.MARSHAL) and pbuild.up_to_date()


@pytest.mark.parametrize("kw", [dict(fails=True), dict(missing=True)])
def test_the_library_is_built_where_the_bindings_part_cannot_be(places, kw):
    places(**kw)
    with pytest.raises(RuntimeError, match="libpkv.so is built, _marshal.so is not"):
        pbuild.build()
    assert os.path.exists(pbuild.LIBRARY) and not os.path.exists(pbuild.MARSHAL) and not pbuild.up_to_date()


def test_without_the_bindings_part_calls_are_marshalled_in_python(monkeypatch):
    monkeypatch.setattr(_lib, "_SHORT", None)
    monkeypatch.delattr(pkv, "_marshal", raising=False)
    monkeypatch.setitem(sys.modules, "paged_kv_prep_gb300._marshal", None)        # importing it raises ImportError
    with pytest.warns(RuntimeWarning, match="_marshal.so is not built"):
        short = _lib._short()
    for name in ("rope_store", "kv4_store", "kv4_load", "kv4_attention", "verify_drafts"):
        assert getattr(short, name)(1, 2) is NotImplemented
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(ValueError, match="CUDA device"):                      # warned once; the Python checks
            pkv.verify_drafts(torch.zeros(3, 100), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                              torch.zeros(3), 2)
