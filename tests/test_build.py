"""The build's order and what makes it run again, with stand-ins for the compilers (no CUDA, no torch headers)."""
import os
import stat

import pytest

from paged_kv_decode_cache_gb300 import build as B

TOUCH = """#!/bin/bash
echo "$0 $*" >> "{log}"
while [ $# -gt 0 ]; do if [ "$1" = -o ]; then echo built > "$2"; fi; shift; done
"""


@pytest.fixture
def tools(tmp_path, monkeypatch):
    """Compilers that only make their output file; the calls of each."""
    log = tmp_path / "calls"
    log.write_text("")
    for name in ("nvcc", "g++"):
        path = tmp_path / "bin" / name
        path.parent.mkdir(exist_ok=True)
        path.write_text(TOUCH.format(log=log))
        path.chmod(path.stat().st_mode | stat.S_IXUSR)
        monkeypatch.setenv({"nvcc": "NVCC", "g++": "CXX"}[name], str(path))
    out = tmp_path / "_build"
    monkeypatch.setattr(B, "BUILD", str(out))
    monkeypatch.setattr(B, "LIB", str(out / "libpagedattn.so"))
    monkeypatch.setattr(B, "BINDING", str(out / "_pa_binding.so"))

    def calls(name):
        lines = log.read_text().splitlines()
        log.write_text("")
        return [x for x in lines if f"/{name} " in x]
    return calls


def test_builds_once(tools):
    B.build()
    assert os.path.exists(B.LIB) and os.path.exists(B.BINDING) and B.up_to_date()
    tools("nvcc")
    B.build()
    assert tools("nvcc") == []


def test_the_library_is_there_when_the_binding_does_not_compile(tools, monkeypatch):
    monkeypatch.setenv("CXX", "/bin/false")
    with pytest.raises(RuntimeError, match="binding"):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING)
    assert not B.up_to_date()
    tools("nvcc")
    with pytest.raises(RuntimeError, match="binding"):
        B.build()
    assert tools("nvcc") == []       # the library is not built again for it
    B.build_library()


def test_the_library_alone_needs_no_torch(tools, monkeypatch):
    monkeypatch.setattr(B, "_compile_binding", lambda: pytest.fail("not asked for"))
    assert B.build_library() == B.LIB and os.path.exists(B.LIB)


def test_another_torch_or_python_builds_the_binding_again(tools, monkeypatch):
    """The binding reads tensors' fields through inlined headers: it fits the torch that it was built with."""
    B.build()
    tools("g++")
    monkeypatch.setattr(B, "binding_abi", lambda: "cpython-999 torch 99.0")
    assert not B.up_to_date() and B.library_up_to_date()
    B.build()
    assert len(tools("g++")) == 1 and tools("nvcc") == []
    assert B.up_to_date()


def test_a_binding_of_another_torch_is_not_loaded(tools, monkeypatch):
    from paged_kv_decode_cache_gb300 import pa
    B.build()
    monkeypatch.setattr(pa, "_native", None)
    monkeypatch.setattr(pa, "lib", lambda: None)
    monkeypatch.setattr(B, "binding_abi", lambda: "cpython-999 torch 99.0")
    with pytest.raises(RuntimeError, match="another torch"):
        pa._binding()
    os.remove(B.BINDING)
    with pytest.raises(RuntimeError, match="missing"):
        pa._binding()


def test_the_abi_names_torch_and_python():
    import sysconfig
    import torch
    assert torch.__version__ in B.binding_abi() and sysconfig.get_config_var("SOABI") in B.binding_abi()
