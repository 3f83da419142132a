"""The entry script: what smoke() reaches, and that running the file ends cleanly."""
import ast
import os
import runpy
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PATH = os.path.join(ROOT, "__graft_entry__.py")


def test_smoke_runs_the_decoding_step():
    with open(PATH) as f:
        tree = ast.parse(f.read())
    smoke = next(n for n in tree.body if isinstance(n, ast.FunctionDef) and n.name == "smoke")
    called = [n.func.id for n in ast.walk(smoke) if isinstance(n, ast.Call) and isinstance(n.func, ast.Name)]
    assert "_smoke_decoding" in called
    assert isinstance(tree.body[-1], ast.If)    # nothing is defined after the script's own run


def test_running_the_script_ends_cleanly(monkeypatch):
    from ulysses_qkv_proj_gb300 import binding, build
    done = []
    monkeypatch.setattr(build, "build", lambda *a, **k: done.append("build"))
    monkeypatch.setattr(binding, "load_library", lambda *a, **k: done.append("load"))
    monkeypatch.setattr(sys, "argv", [PATH])
    runpy.run_path(PATH, run_name="__main__")
    assert done == ["build", "load"]
