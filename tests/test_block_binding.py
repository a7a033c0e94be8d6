"""The CPython extension that makes ordinary calls: it belongs to the Python that
built it, and the package works without it (no GPU needed)."""
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

from conftest import ROOT
from test_train_args import mp  # noqa: F401


def load_build():
    sys.path.insert(0, ROOT)
    import __graft_entry__
    return __graft_entry__._load_by_path("mp_lib_build_again", "mixed_precision_adamw_gb300/build.py")


def test_the_name_tells_the_interpreter(mp):  # noqa: F811
    from mixed_precision_adamw_gb300 import _binding
    assert _binding.__file__.endswith("_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
    assert not os.path.exists(os.path.join(os.path.dirname(_binding.__file__), "_binding.so"))  # any Python's


def test_another_interpreters_is_not_counted(mp, monkeypatch):  # noqa: F811
    assert not load_build().is_stale()
    ask = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda k: ".cpython-999-any.so" if k == "EXT_SUFFIX" else ask(k))
    assert load_build().is_stale()


@pytest.mark.parametrize("missing", ["compiler", "headers"])
def test_what_builds_it_may_be_missing(mp, missing, monkeypatch, tmp_path, capsys):  # noqa: F811
    b = load_build()
    before = os.path.getmtime(b.BINDING)
    if missing == "compiler":
        which = shutil.which
        monkeypatch.setattr(shutil, "which", lambda n, *a, **k: None if n in ("gcc", "cc") else which(n, *a, **k))
    else:
        paths = sysconfig.get_paths
        monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: {**paths(*a, **k), "include": str(tmp_path)})
    b._binding()
    assert "_binding" in capsys.readouterr().err
    assert os.path.getmtime(b.BINDING) == before
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "none.so"))
    assert not b.is_stale()  # nothing that could be built is missing


def test_the_package_without_it(mp, tmp_path):  # noqa: F811
    here = os.path.join(ROOT, "mixed_precision_adamw_gb300")
    to = tmp_path / "mixed_precision_adamw_gb300"
    to.mkdir()
    for f in os.listdir(here):
        if f.endswith(".py"):
            shutil.copy(os.path.join(here, f), to / f)
    os.symlink(os.path.join(here, "libmpadamw.so"), to / "libmpadamw.so")
    code = """
import torch
import mixed_precision_adamw_gb300 as mp
torch.cuda.current_device = lambda: 0
x = torch.zeros(4, 64, dtype=torch.bfloat16)
q = torch.zeros(4, 64, dtype=torch.uint8)
t = torch.zeros(8, dtype=torch.int64)
rstd = torch.zeros(4)
for call in (lambda: mp.mp_rmsnorm_forward(x.clone(), x), lambda: mp.mp_rmsnorm_backward(x, None, x, x, None, rstd),
             lambda: mp.mp_gated_forward(x.clone(), x), lambda: mp.mp_gated_backward(x, None, x, x),
             lambda: mp.mp_pack8(q, rstd, x), lambda: mp.mp_unpack8(x, q, rstd),
             lambda: mp.mp_rope(x[None], x[None], None, None, t)):
    try:
        call()
    except ValueError as e:
        assert "CUDA tensor" in str(e), e
    else:
        raise AssertionError("not refused")
assert mp.mp_rope_frequencies(64, device="cpu")[0].numel() == 32
print("fine")
"""
    env = {**os.environ, "PYTHONPATH": str(tmp_path)}
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, env=env, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr


def test_an_outdated_one_goes(mp, monkeypatch, tmp_path):  # noqa: F811
    # its calls may not be the library's any more
    b = load_build()
    old = tmp_path / "old.so"
    old.write_bytes(b"")
    os.utime(old, (1, 1))
    monkeypatch.setattr(b, "BINDING", str(old))
    monkeypatch.setattr(b, "_binding_needs", lambda: "a C compiler")
    b._binding()
    assert not old.exists()
