"""CPU: the C library is built and linked whether or not the Python module beside it can be."""
import pytest

from dequant_gemm_amd import build as B


@pytest.fixture
def steps(monkeypatch, tmp_path):
    """Build steps recorded instead of run."""
    done = []
    for name in ("LIB", "BENCH_LIB", "HOST_LIB"):
        monkeypatch.setattr(B, name, str(tmp_path / name))
    monkeypatch.setattr(B, "OBJDIR", str(tmp_path))
    monkeypatch.setattr(B, "_compile", lambda src, asm, objdir=None: str(tmp_path / src))

    def run(cmd):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        done.append(out)
    monkeypatch.setattr(B, "_run", run)
    return done, tmp_path


def test_everything(steps):
    done, path = steps
    assert B.build(verbose=False) == str(path / "LIB")
    assert all((path / n).exists() for n in ("LIB", "BENCH_LIB", "HOST_LIB"))


@pytest.mark.parametrize("part", ["_compile_host", "_link_host"])
def test_no_host_compiler(steps, monkeypatch, part):
    done, path = steps

    def missing(*_):
        raise FileNotFoundError("g++")
    monkeypatch.setattr(B, part, missing)
    with pytest.raises(RuntimeError, match=r"_host.*libnf4|libnf4.*_host"):
        B.build(verbose=False)
    assert (path / "LIB").exists() and (path / "BENCH_LIB").exists() and not (path / "HOST_LIB").exists()
