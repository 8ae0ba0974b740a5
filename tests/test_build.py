"""The build step's choices, with the compilers replaced by a record of their
commands (no GPU, nothing is compiled)."""
import os

import pytest

from paged_kv_cache_174_gb300 import build as pkg_build


@pytest.fixture
def commands(tmp_path, monkeypatch):
    """Builds go to an empty folder; the list holds the commands of each."""
    out = tmp_path / "_build"
    monkeypatch.setattr(pkg_build, "OUT_DIR", str(out))
    monkeypatch.setattr(pkg_build, "LIB", str(out / pkg_build.LIB_NAME))
    monkeypatch.setattr(pkg_build, "BINDING", str(out / pkg_build.BINDING_NAME))
    ran = []

    def run(cmd, verbose):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(pkg_build, "_run", run)
    return ran


def test_library_is_built_where_there_is_no_torch(commands, monkeypatch, capsys):
    find = pkg_build.importlib.util.find_spec
    monkeypatch.setattr(pkg_build.importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else find(name, *a))
    assert pkg_build.build() == pkg_build.LIB and os.path.exists(pkg_build.LIB)
    assert len(commands) == len(pkg_build.SOURCES) + 1  # each source, and the library
    assert not os.path.exists(pkg_build.BINDING)
    assert "torch not found" in capsys.readouterr().err


def test_extension_is_built_again_for_another_torch(commands, tmp_path, monkeypatch):
    fake = tmp_path / "torch"
    fake.mkdir()
    (fake / "version.py").write_text("__version__ = '2.9.1'\n")
    monkeypatch.setattr(pkg_build, "_torch_dir", lambda: str(fake))
    pkg_build.build()
    assert os.path.exists(pkg_build.BINDING)
    commands.clear()
    pkg_build.build()
    assert commands == []  # nothing changed
    (fake / "version.py").write_text("__version__ = '2.11.0'\n")
    pkg_build.build()
    outputs = [os.path.basename(c[c.index("-o") + 1]) for c in commands]
    assert "pa_binding.o" in outputs and pkg_build.BINDING_NAME + ".tmp" in outputs
    assert not any(c[c.index("-o") + 1].endswith(".o") for c in commands
                   if "pa_binding" not in c[c.index("-o") + 1])  # no kernel again
    commands.clear()
    pkg_build.build()
    assert commands == []
