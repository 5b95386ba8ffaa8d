"""The binding's native module (_call.so): when it is loaded.  Host-only."""

import os
import subprocess
import sys

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
