"""The build script: what it builds where, and when it builds again."""
import subprocess
import sys

import pytest
import torch

from bigvgan_waveform_decoder_alias_b200 import build_native


@pytest.fixture(scope="module")
def built():
    build_native.build()


@pytest.fixture
def commands(built, monkeypatch):
    """The compilers' command lines, none of them run."""
    ran = []
    monkeypatch.setattr(subprocess, "check_call", lambda cmd, **kw: ran.append(cmd))
    monkeypatch.setattr(build_native.os, "replace", lambda a, b: None)
    return ran


def test_the_library_is_built_without_torch(commands, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)  # as where it is not installed
    assert build_native.build(force=True) == build_native.LIB
    assert len(commands) == 1 and build_native.LIB + ".tmp" in commands[0]
    assert "no torch" in capsys.readouterr().err


def test_the_library_is_built_before_the_binding(commands):
    build_native.build(force=True)
    assert [c[c.index("-o") + 1] for c in commands] == [build_native.LIB + ".tmp",
                                                        build_native.BINDING + ".tmp"]


def test_the_binding_follows_the_torch_it_was_built_against(commands, monkeypatch):
    build_native.build_binding()
    assert commands == []  # up to date
    monkeypatch.setattr(torch, "__version__", "1.2.3")
    build_native.build_binding()
    assert len(commands) == 1 and build_native.BINDING + ".tmp" in commands[0]
