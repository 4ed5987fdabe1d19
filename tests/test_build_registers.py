"""The build ends where a kernel that moves registers between its warps has not the count that the split adds up to.  CPU only."""
import pytest

from newton_solve_nonlinear_b200 import build

ENTRY = """ptxas info    : Compiling entry function '{name}' for 'sm_100a'
ptxas info    : Function properties for {name}
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used {used} registers, used 3 barriers
ptxas info    : Compile time = 1.000 ms
"""
SPLIT, OTHER = "_ZN7pararnn12_GLOBAL__N_118ss_backward_kernelIfLi2ELi8ELb1EEEvNS_6SsArgsE", "_ZN7pararnn14ss_join_kernelEv"


@pytest.mark.parametrize("used,fits", [(128, True), (120, False), (127, False), (168, False)])
def test_a_split_needs_its_exact_count(used, fits):
    log = ENTRY.format(name=OTHER, used=40) + ENTRY.format(name=SPLIT, used=used) + ENTRY.format(name=OTHER, used=32)
    if fits:
        build.check_registers(log)
    else:
        with pytest.raises(RuntimeError, match=f"{used} registers"):
            build.check_registers(log)


def test_other_kernels_may_have_any():
    build.check_registers("".join(ENTRY.format(name=OTHER, used=n) for n in (16, 100, 255)))


def test_a_source_that_fails_leaves_no_object(tmp_path, monkeypatch):
    """A later build would take it for up to date."""
    class Result:
        returncode, stdout, stderr = 0, "", ENTRY.format(name=SPLIT, used=120)

    src = tmp_path / "kernel.cu"
    src.write_text("")
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: (tmp_path / "kernel.o").write_text("") or Result)
    (tmp_path / "kernel.o").unlink(missing_ok=True)
    with pytest.raises(RuntimeError, match="registers"):
        build._compile(str(src), False)
    assert not (tmp_path / "kernel.o").exists()
