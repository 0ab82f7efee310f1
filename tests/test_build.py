"""The build step without what only the native part of the Python binding needs: the C library is built all the same."""
import os
import sys

import pytest

from fp8_block_scaled_05_amd import build


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """Compilers that write their output file and note their commands; nothing is compiled."""
    commands = []

    def run(cmd, verbose):
        if cmd[0] == "g++" and not available["g++"]:
            raise FileNotFoundError("g++")
        commands.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    available = {"g++": True}
    which = build.shutil.which
    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "hipcc", lambda: "hipcc")
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libfp8bs.so"))
    monkeypatch.setattr(build, "MARSHAL_PATH", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(build.shutil, "which", lambda name: None if name == "g++" and not available["g++"] else which(name))
    return commands, available, tmp_path


def test_all_is_built(fake):
    pytest.importorskip("torch")
    commands, _, where = fake
    assert build.build() == str(where / "libfp8bs.so")
    assert sorted(os.listdir(where)) == ["_marshal.so", "libfp8bs.so"]
    assert len(commands) == len(build.SOURCES) + 2 and commands[-1][0] == "g++"


@pytest.mark.parametrize("missing", ["torch", "g++"])
def test_the_library_is_built_without_the_binding(fake, missing, monkeypatch, capsys):
    commands, available, where = fake
    if missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    else:
        available["g++"] = False
    (where / "_marshal.so").write_text("of an older build")
    assert build.build() == str(where / "libfp8bs.so")
    assert os.listdir(where) == ["libfp8bs.so"]        # an older module would not fit the library
    assert all(c[0] == "hipcc" for c in commands)
    assert missing in capsys.readouterr().out


def test_a_missing_native_module_is_named(monkeypatch, tmp_path):
    import fp8_block_scaled_05_amd as fb
    from fp8_block_scaled_05_amd import decoder
    pytest.importorskip("torch")
    monkeypatch.setattr(decoder, "_marshal", decoder._Unloaded())
    monkeypatch.setattr(decoder, "MARSHAL_PATH", str(tmp_path / "_marshal.so"))
    with pytest.raises(ImportError, match="_marshal.so is missing: build it"):
        fb.fp8_moe_route(None, 2)
