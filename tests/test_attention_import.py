"""The package without torch or without the compiled module of the attention calls (no GPU needed).

Only an attention plan needs torch, and none needs the module, which saves
host time: importing the package loads neither.
"""
import importlib.util
import os
import shutil
import subprocess
import sys
import textwrap

import pytest

import fusion_b2b_gemm_gb300 as b2b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "fusion_b2b_gemm_gb300")


def python(code, root=ROOT):
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=root, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": root})
    assert r.returncode == 0, r.stderr
    return r.stdout


def test_import_does_not_load_torch():
    out = python("""
        import sys
        import fusion_b2b_gemm_gb300 as b2b
        print("torch" in sys.modules, hasattr(b2b, "PromptAttentionPlan"))
        """)
    assert out.split() == ["False", "True"]


def test_import_without_torch():
    out = python("""
        import sys
        sys.modules["torch"] = None
        from fusion_b2b_gemm_gb300 import *
        print(b2b_status_string(0).decode(), Plan.__name__, GemmPlan.__name__)
        try:
            PromptAttentionPlan("f16", 4, 2, 64)
        except ImportError as e:
            print("torch" in str(e))
        """)
    assert out.split("\n")[1] == "True" and "Plan GemmPlan" in out


@pytest.mark.parametrize("there", ["missing", "damaged", "for another torch"])
def test_without_the_compiled_module(tmp_path, there):
    pytest.importorskip("torch")
    copy = tmp_path / "fusion_b2b_gemm_gb300"
    shutil.copytree(PACKAGE, copy, ignore=shutil.ignore_patterns("_lib", "_build", "csrc", "__pycache__"))
    (copy / "_lib").mkdir()
    os.symlink(b2b.library_path(), copy / "_lib" / "libb2b.so")
    if there == "damaged":
        (copy / "_lib" / "attn_binding.so").write_bytes(b"not a module")
    if there == "for another torch":
        os.symlink(os.path.join(os.path.dirname(b2b.library_path()), "attn_binding.so"), copy / "_lib" / "attn_binding.so")
    out = python(f"""
        import warnings
        import fusion_b2b_gemm_gb300 as b2b
        from fusion_b2b_gemm_gb300 import attention
        print(b2b.b2b_status_string(0).decode())
        import torch
        if {there == "for another torch"}:
            torch.__version__ = "0.0.1"
        with warnings.catch_warnings(record=True) as seen:
            warnings.simplefilter("always")
            attention._load()
        print([w.category.__name__ for w in seen if "attn_binding.so" in str(w.message)])
        print(attention._binding.bind(0, True, 4, 2, 64, 0), attention._binding.prompt(None, 0), attention._binding.shared(None, 0))
        """, str(tmp_path))
    assert out.split("\n")[1:3] == ["['RuntimeWarning']", "None None None"]


def test_build_without_torch(monkeypatch):
    spec = importlib.util.spec_from_file_location("_b2b_build_test", os.path.join(PACKAGE, "_build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    assert build.build_binding() is None
