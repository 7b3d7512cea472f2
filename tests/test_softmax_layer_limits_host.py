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


# ----------------------------------------- outputs that a call still reads
# bf16, 4 tokens, 8 query and 2 key-value heads of 64; every array in a place of its own
AT = {n: A * (i + 1) for i, n in enumerate("q k v qo ko dqo dko dq dk dqw dkw w table pos kc vc slots bt "
                                           "lens out ws".split())}


def _call(lib, name, at):
    p = {**AT, **{n: AT[o] for n, o in at.items()}}
    rot, shape = [p["pos"], p["table"], 64, 64, 0, p["w"], p["w"], 1e-6], [4, 8, 2, 64, la.LA_DTYPE_BF16]
    q, k, v = [p["q"], 512], [p["k"], 128], [p["v"], 128]
    cache = [p["kc"], 2048, p["vc"], 2048]
    args = {
        "qk_norm_rope": q + k + rot + shape + [p["qo"], 512, p["ko"], 128, None],
        "qk_norm_rope_backward": q + k + rot + shape + [p["dqo"], 512, p["dko"], 128, p["dq"], 512, p["dk"],
                                                        128, p["dqw"], p["dkw"], p["ws"], 1 << 30, None],
        "paged_append": q + k + v + rot + shape + [p["qo"], 512] + cache + [p["slots"], 10, 16, None],
        "paged_step": q + k + v + rot + cache + [p["slots"], p["bt"], 5, 5, p["lens"], 10, 16] + shape +
        [0.1, p["out"], None, p["ws"], 1 << 30, None],
    }[name]
    return getattr(lib, "lightning_attn_" + name)(*args)


@pytest.mark.parametrize("name, at", [
    ("qk_norm_rope", dict(qo="k")), ("qk_norm_rope", dict(ko="q")), ("qk_norm_rope", dict(ko="qo")),
    ("qk_norm_rope_backward", dict(dq="k")), ("qk_norm_rope_backward", dict(dk="q")),
    ("qk_norm_rope_backward", dict(dq="dko")), ("qk_norm_rope_backward", dict(dk="dqo")),
    ("qk_norm_rope_backward", dict(dkw="dqw")),
    ("paged_append", dict(qo="k")), ("paged_append", dict(qo="v")), ("paged_append", dict(vc="kc")),
    ("paged_step", dict(vc="kc"))])
def test_outputs_over_other_arguments_are_refused(lib, name, at):
    assert _call(lib, name, at) == la.LA_ERR_INVALID_ARG
    assert " one array" in lib.lightning_attn_last_error().decode() or \
        any(w in lib.lightning_attn_last_error().decode() for w in ("other", "aliases", "q_out is"))


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
