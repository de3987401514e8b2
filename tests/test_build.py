"""What the build needs and in which order it works (nothing is compiled here)."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

from gated_delta_rule_62_amd import _build


@pytest.fixture()
def commands(monkeypatch):
    """The build's commands and finished files, recorded instead of run."""
    seen = []

    def run(cmd, **kw):
        seen.append([os.path.basename(c) for c in cmd])

    monkeypatch.setattr(_build.subprocess, "run", run)
    monkeypatch.setattr(_build.os, "replace", lambda a, b: seen.append(["done",
                                                                        os.path.basename(b)]))
    return seen


def test_the_library_is_first_and_needs_rocm_alone(commands, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    assert _build.build() == _build.LIB_PATH
    assert [c[c.index("-c") + 1] for c in commands if "-c" in c] == _build.SOURCES
    assert commands[-1] == ["done", "libkda.so"]
    assert {c[0] for c in commands[:-1]} == {"hipcc"}


def test_the_calls_from_python_follow(commands, monkeypatch):
    _build.build()
    assert commands.index(["done", "libkda.so"]) < len(commands) - 2
    assert "serving_calls.cpp" in commands[-2] and commands[-2][0] == "amdclang++"
    assert commands[-1] == ["done", "_serving_calls.so"]
    # a failure there leaves the library in place and is reported
    ran = _build.subprocess.run

    def fail(cmd, **kw):
        ran(cmd, **kw)
        if "serving_calls.cpp" in commands[-1]:
            raise subprocess.CalledProcessError(1, cmd)

    commands.clear()
    monkeypatch.setattr(_build.subprocess, "run", fail)
    with pytest.raises(subprocess.CalledProcessError):
        _build.build()
    assert ["done", "libkda.so"] in commands
