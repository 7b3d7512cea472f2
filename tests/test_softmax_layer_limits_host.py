"""Softmax-layer operators without a GPU: refusals and builds at the edges of
their contracts."""
import subprocess
import sys

import pytest

import lightning_attention_attn_gb300 as la
from lightning_attention_attn_gb300 import build as labuild

A = 0x100000  # an aligned fake address: validation fails before any use


@pytest.fixture(scope="module")
def lib():
    return la.load(labuild.build())


@pytest.mark.parametrize("lens_out, count_out", [(A, A + 0x100), (A + 0x100, A)])
def test_paged_reserve_refuses_new_lens_as_an_output(lib, lens_out, count_out):
    a = 2 * A
    status = lib.lightning_attn_paged_reserve(a, 5, 5, a, A, None, 4, a, a, 10, 16, 4, a, a, a, a,
                                              lens_out, count_out, None)
    assert status == la.LA_ERR_INVALID_ARG
    assert "new_lens" in lib.lightning_attn_last_error().decode()


def test_library_builds_without_torch():
    """The C library needs neither torch nor the package (which imports it)."""
    path = labuild.build()
    code = ("import runpy, sys; sys.modules['torch'] = None; "
            f"print(runpy.run_path({labuild.__file__!r})['build']())")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == path


def test_library_is_in_place_where_the_binding_cannot_be_built(tmp_path, monkeypatch):
    ran = []

    def run(cmd, what):
        ran.append(what)
        if what == "binding":
            raise RuntimeError("no Python headers")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return ""

    monkeypatch.setattr(labuild, "_run", run)
    for name in ("BUILD_DIR", "LIB_PATH", "BINDING_PATH"):
        monkeypatch.setattr(labuild, name, str(tmp_path / getattr(labuild, name).split("/")[-1])
                            if name != "BUILD_DIR" else str(tmp_path))
    for _ in range(2):
        with pytest.raises(RuntimeError, match="no Python headers"):
            labuild.build()
        assert (tmp_path / labuild.LIB_NAME).exists()
    assert ran.count("link") == 1  # the second build found the library up to date
    monkeypatch.setattr(labuild, "_run", lambda cmd, what: open(cmd[cmd.index("-o") + 1], "w").close())
    labuild.build()
    assert (tmp_path / "_lightning_binding.so").exists()
