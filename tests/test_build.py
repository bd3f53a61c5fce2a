"""The build: the same code whatever machine builds it."""
import os

import bench
from entropy_loss_gb300 import build


def test_code_does_not_depend_on_the_number_of_cpus(monkeypatch):
    """nvcc's split compilation gives most kernels other registers with another
    number of parts (one per CPU when it is 0)."""
    cmds = []
    for n in (2, 64):
        monkeypatch.setattr(os, "cpu_count", lambda n=n: n)
        cmds.append(build.command("out.so"))
    assert cmds[0] == cmds[1]
    assert not any("split-compile" in a for a in cmds[0])


def test_command_and_digest_follow_the_flags(monkeypatch):
    before = bench.kernel_sources_digest()
    monkeypatch.setattr(build, "FLAGS", build.FLAGS + ["--use_fast_math"])
    assert "--use_fast_math" in build.command("out.so")
    assert bench.kernel_sources_digest() != before


def test_a_changed_command_rebuilds():
    assert build.__file__ in build.sources()
