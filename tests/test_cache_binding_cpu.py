"""The CPython module is a shorter way and never the only one: a file that does not load, or that was built for another
library or another torch, leaves the calls to ctypes; and one that cannot be rebuilt does not stay."""
import subprocess
import sys

import pytest
import torch

import attention_forward_02_gb300 as fa
from attention_forward_02_gb300 import build, cache


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build_library()
    return fa.load()


@pytest.fixture
def fresh(monkeypatch):
    """The module not looked for yet."""
    monkeypatch.setattr(cache, "_module", None)
    monkeypatch.setattr(cache, "_bound", None)


def refused_as_ever():
    """A call goes through: here to the refusal of CPU tensors."""
    c = fa.FACache.empty(4, 2, 16, 32, device="cpu")
    with pytest.raises(fa.FAError):
        fa.fa_cache_read(c, torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), 5)


def compile_as(tmp_path, change):
    """The module built by the usual command but for a changed definition."""
    out = str(tmp_path / "binding.so")
    command = build.binding_command(out)
    at = [i for i, x in enumerate(command) if x.startswith(change[0])]
    assert at, "the command names no %s" % change[0]
    for i in at:
        command[i] = change[1]
    subprocess.run(command, check=True)
    return out


def test_the_built_module_is_used(fresh):
    assert build.build_binding() == build.BINDING
    assert cache._quick()
    refused_as_ever()


@pytest.mark.parametrize("what", ["text", "empty", "another library"])
def test_a_file_that_does_not_load(fresh, monkeypatch, tmp_path, what):
    path = tmp_path / "binding.so"
    path.write_bytes(b"no library" if what == "text" else b"")
    if what == "another library":  # loads, but is no such module
        (tmp_path / "x.c").write_text("int x;")
        subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(path), str(tmp_path / "x.c")], check=True)
    monkeypatch.setattr(cache, "BINDING", str(path))
    assert not cache._quick()
    refused_as_ever()


def test_a_module_for_another_abi(fresh, monkeypatch):
    assert cache._quick()

    class Other:  # the library, one version on
        def __getattr__(self, name):
            return getattr(fa.load(), name)

        def fa_abi_version(self):
            return fa.fa_abi_version() + 1

    other = Other()
    monkeypatch.setattr(cache, "load", lambda: other)
    assert not cache._quick()
    refused_as_ever()


def test_a_module_for_another_torch(fresh, monkeypatch, tmp_path):
    path = compile_as(tmp_path, ("-DFA_TORCH_VERSION=", '-DFA_TORCH_VERSION="1.0.0+other"'))
    monkeypatch.setattr(cache, "BINDING", path)
    assert not cache._quick()
    refused_as_ever()


def test_a_stale_module_does_not_stay(monkeypatch, tmp_path):
    path = tmp_path / "binding.so"
    path.write_bytes(b"built from older sources")
    monkeypatch.setattr(build, "BINDING", str(path))
    monkeypatch.setattr(build, "binding_command", lambda out: [sys.executable, "-c", "raise SystemExit(1)"])
    assert build.build_binding(force=True) is None
    assert not path.exists()


def test_another_torch_makes_it_stale(monkeypatch, tmp_path):
    path = tmp_path / "binding.so"
    built = []

    def command(out):
        built.append(out)
        return [sys.executable, "-c", "open(%r, 'w').write('built')" % out]

    monkeypatch.setattr(build, "BINDING", str(path))
    monkeypatch.setattr(build, "binding_command", command)
    assert build.build_binding() == str(path) and len(built) == 1
    assert build.build_binding() == str(path) and len(built) == 1
    monkeypatch.setattr(torch, "__version__", "1.0.0+other")
    assert build.build_binding() == str(path) and len(built) == 2
