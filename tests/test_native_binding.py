"""The binding's native module (_call.so): when it is loaded.  Host-only."""

import os
import subprocess
import sys

from block_sparse_attention_psa_b200 import build, psa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code, **env):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, env={**os.environ, **env})
    assert r.returncode == 0, r.stderr
    return r.stdout


def test_importing_loads_no_library_of_this_repository():
    """Neither the binding's import nor the benchmark's (whose reference arm runs
    on the host cores alone) maps a library; the first use loads both."""
    out = run("""
import bench
from block_sparse_attention_psa_b200 import psa
mapped = lambda: {x.split('/')[-1].strip() for x in open('/proc/self/maps') if 'block_sparse' in x}
print(sorted(mapped()))
assert psa._native is not None
print(sorted(mapped()))
""")
    assert out.split("\n")[:2] == ["[]", "['_call.so', 'libpsa.so']"]


def test_the_first_serving_call_loads_it():
    out = run("""
import torch
from block_sparse_attention_psa_b200 import psa
q, k = torch.zeros(1, 1, 1, 64).half(), torch.zeros(1, 1, 8, 64).half()
for call in (lambda: psa.psa_decode(q, k, k), lambda: psa.psa_key_weight(q, k, torch.zeros(1, 1, 1)),
             lambda: psa.psa_cache_evict(k, k, torch.zeros(1, 1, 8), 2)):
    try:
        call()
    except ValueError as e:
        print(e)
print(psa._native.__name__)
""")
    assert out.split("\n") == 3 * ["tensor must live on a CUDA device"] + ["block_sparse_attention_psa_b200._call", ""]


def test_it_serves_only_the_pytorch_it_was_built_for(monkeypatch):
    assert psa._native is not None and psa._native.built_for == build.built_for()
    monkeypatch.setattr(build, "built_for", lambda: "torch 9.9.9 cpython-399")
    assert psa._load_native() is None


def test_another_pytorch_builds_it_anew(monkeypatch, tmp_path):
    """Whatever the files' times say."""
    made = []

    def compiler(cmd, **kw):
        made.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "CALL", str(tmp_path / "_call.so"))
    monkeypatch.setattr(build, "CALL_STAMP", str(tmp_path / "stamp"))
    monkeypatch.setattr(build.subprocess, "run", compiler)
    build._build_call()
    build._build_call()
    assert len(made) == 1
    monkeypatch.setattr(build, "built_for", lambda: "torch 9.9.9 cpython-399")
    build._build_call()
    build._build_call()
    assert len(made) == 2 and any("torch 9.9.9 cpython-399" in x for x in made[1])
