"""The build on the CPU, with the compilers replaced: what comes out when a
part of it cannot be built."""

import os
import subprocess
import sys

import pytest

import bit_grouped_moe_amd as gq
import bit_grouped_moe_amd.build as build


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """Build into tmp_path.  hipcc writes its output file and succeeds; the
    host compiler does as `state["host"]` says; returns (state, tmp_path)."""
    state = {"host": "ok", "hip": "ok"}

    def run(cmd, **kw):
        host = "hipcc" not in os.path.basename(cmd[0])
        how = state["host" if host else "hip"]
        if how == "absent":
            raise FileNotFoundError(cmd[0])
        if how == "fails":
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("new")
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(build.subprocess, "run", run)
    for name, file in (("BUILD", "objects"), ("LIB", "libgq.so"), ("PROBE_LIB", "libgq_probes.so"),
                       ("CALLS_LIB", "_calls.so")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    return state, tmp_path


def test_whole_build(fake):
    state, d = fake
    assert build.build() == str(d / "libgq.so")
    for f in ("libgq.so", "libgq_probes.so", "_calls.so"):
        assert (d / f).read_text() == "new"


@pytest.mark.parametrize("how", ["absent", "fails", "no torch"])
def test_libraries_without_the_short_calls(fake, how, capsys, monkeypatch):
    """No host compiler, no headers for it or no torch: the kernels are built
    all the same, an earlier module goes, and the reason is printed."""
    state, d = fake
    if how == "no torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    state["host"] = how
    (d / "_calls.so").write_text("old")
    assert build.build() == str(d / "libgq.so")
    assert (d / "libgq.so").read_text() == "new" and (d / "libgq_probes.so").read_text() == "new"
    assert not (d / "_calls.so").exists()
    assert "short calls" in capsys.readouterr().err


def test_kernels_that_do_not_compile_end_the_build(fake):
    state, d = fake
    state["hip"] = "fails"
    with pytest.raises(RuntimeError, match="no such header"):
        build.build()
    assert not (d / "libgq.so").exists()


def test_short_calls_of_another_header_are_not_used(monkeypatch, tmp_path):
    """A module that was built with other declarations would hand the library
    arguments that it does not take; other comments change nothing."""
    lib = gq.load_library()
    assert gq._calls is not None
    with open(build.HEADER) as f:
        text = f.read()
    header = tmp_path / "gq.h"
    monkeypatch.setattr(build, "HEADER", str(header))
    try:
        for there, used in ((text, True), ("/* more words */" + text, True), (None, False),
                            (text.replace("int32_t topk", "int64_t topk"), False),
                            (text.replace("int32_t renormalize; ", "int32_t renormalize, more; "),
                             False)):
            header.unlink(missing_ok=True)
            if there is not None:
                header.write_text(there)
                assert used == (there.endswith(text))
            gq._load_calls(lib)
            assert (gq._calls is not None) == used
    finally:
        monkeypatch.undo()
        gq._load_calls(lib)
    assert gq._calls is not None
