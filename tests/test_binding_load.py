"""Loading of the compiled marshalling (no GPU): the calls that do not need it
work without it, those that do say why each time."""
import os
import sysconfig

import pytest

from mla_decode_attention_07_gb300 import build, libmla


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return libmla.load()


def _append():
    torch = pytest.importorskip("torch")
    bf, i32 = torch.bfloat16, torch.int32
    libmla.mla_rope_append(torch.zeros(1, 1, 576, dtype=bf), torch.zeros(1, 64, 1, 576, dtype=bf),
                           torch.zeros(1, 1, dtype=i32), torch.zeros(1, dtype=i32),
                           torch.zeros(64, 64), stream=0)


@pytest.mark.parametrize("what", ["missing", "broken"])
def test_library_loads_without_the_module(lib, monkeypatch, tmp_path, what):
    path = tmp_path / build.BINDING
    if what == "broken":
        path.write_bytes(b"no module")
    monkeypatch.setattr(libmla, "_lib", None)
    monkeypatch.setattr(libmla, "_binding", None)
    monkeypatch.setattr(libmla, "BINDING_PATH", str(path))
    assert libmla.load().mla_decode_plan is not None
    assert libmla.mla_plan_size_for_clusters(1, 1, 16, 76) > 0
    for _ in range(2):                                   # not only the first time
        with pytest.raises(RuntimeError, match="compiled marshalling"):
            _append()
    monkeypatch.setattr(libmla, "BINDING_PATH", os.path.join(build.OUT_DIR, build.BINDING))
    with pytest.raises(libmla.MlaError, match="current CUDA device"):
        _append()                                        # once it is there, it is found


def test_module_is_this_pythons(lib):
    assert build.BINDING.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert os.path.exists(libmla.BINDING_PATH)


def test_build_without_python_headers_leaves_the_module_out(monkeypatch, tmp_path):
    """No module is asked for and none compiled where Python.h is missing."""
    monkeypatch.setattr(build.sysconfig, "get_paths",
                        lambda: {"include": str(tmp_path), "platinclude": str(tmp_path)})
    assert build.python_includes() is None
    lib, calls = tmp_path / "libmla.so", []

    class Done:
        returncode = 0

        def communicate(self):
            return "", None

    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(lib))
    monkeypatch.setattr(build.subprocess, "Popen", lambda cmd, **kw: calls.append(cmd) or Done())
    monkeypatch.setattr(build.subprocess, "check_call",
                        lambda cmd: open(cmd[cmd.index("-o") + 1], "w").close())
    assert build.build() == str(lib) and lib.exists()
    assert len(calls) == len(build.SOURCES) and not any("binding.c" in c[-3] for c in calls)
    assert build.build() == str(lib) and len(calls) == len(build.SOURCES)     # up to date
