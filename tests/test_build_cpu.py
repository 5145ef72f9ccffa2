"""What a build leaves behind: the library alone serves the recurrence's calls, and the torch binding is taken for
built only where it was built for the torch that is there (CPU)."""
import os
import shutil
import subprocess
import sys

import pytest

PKG = "linear_attention_state_recurrent_gb300"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def build():
    from linear_attention_state_recurrent_gb300 import build as b
    b.build()
    return b


@pytest.fixture
def without_binding(build, tmp_path):
    """The package with libkda.so and no torch binding, in a folder of its own."""
    os.makedirs(tmp_path / PKG)
    for f in ("__init__.py", "build.py", "kda.py", "libkda.so"):
        shutil.copy(os.path.join(ROOT, PKG, f), tmp_path / PKG / f)
    return tmp_path


def run(folder, code):
    return subprocess.run([sys.executable, "-c", code], cwd=folder, capture_output=True, text=True, timeout=300,
                          env=dict(os.environ, PYTHONPATH=str(folder)))


def test_the_recurrences_calls_need_no_torch_binding(without_binding):
    r = run(without_binding, f"""
from {PKG} import kda
assert kda.__file__.startswith({str(without_binding)!r})
assert kda.lib.kda_selftest_bounded_wait(None, None) == 1 and "err_flags" in kda.last_error()
assert kda.kda_chunk_prefill_workspace_bytes(__import__("torch").tensor([0, 64]), 2, 128, 128) > 0
print("there")
""")
    assert r.returncode == 0 and "there" in r.stdout, r.stderr[-2000:]


def test_a_call_that_needs_the_torch_binding_says_so(without_binding):
    r = run(without_binding, f"""
import torch
from {PKG} import kda
try:
    kda.kda_norm_quant(torch.zeros(2, 128))
except RuntimeError as e:
    print("said:", e)
""")
    assert r.returncode == 0 and "not built" in r.stdout and "build()" in r.stdout, r.stderr[-2000:]


def test_a_binding_that_does_not_compile_leaves_the_library(build, monkeypatch, tmp_path):
    def fails():
        raise RuntimeError("no headers")
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libkda.so"))
    monkeypatch.setattr(build, "_compile_binding", fails)
    monkeypatch.setattr(build, "OBJ", str(tmp_path / "obj"))
    small = tmp_path / "one.cu"
    small.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(build, "_sources", lambda: [str(small)])
    with pytest.raises(RuntimeError, match="no headers"):
        build.build(force=True)
    assert os.path.exists(build.LIB)


def test_a_binding_of_another_torch_is_not_taken_for_built(build, monkeypatch):
    from linear_attention_state_recurrent_gb300 import kda
    assert build.up_to_date()
    here = build.binding_lib()
    real = build.importlib.metadata.version
    monkeypatch.setattr(build.importlib.metadata, "version", lambda name: "1.0" if name == "torch" else real(name))
    assert build.binding_lib() != here and not build.up_to_date()
    with pytest.raises(RuntimeError, match="not built for this torch"):
        kda._TorchBinding().norm_quant
    monkeypatch.undo()
    assert build.up_to_date()
