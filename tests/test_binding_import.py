"""The package without its compiled module (built against one interpreter and
one PyTorch): what does not need it works (no GPU needed)."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import os, sys
{before}
import mla_latent_kv_uk_gb300 as m
assert m.mla_status_string(1) == "invalid argument"
assert m.mla_decode_workspace_size(2, 1, 128, 4096) > 0
assert m.mla_decode_window_workspace_size(2, 1, 128, 640000) > 0
assert "_mla_binding" not in sys.modules
import torch
cpu = torch.zeros((2, 1, 4, 576), dtype=torch.bfloat16)
for call in (lambda: m.mla_decode_paged_window(cpu, cpu[0], None, None, sm_scale=1.0, window=0),
             lambda: m.mla_rope_cache_append(None, cpu, cpu, cpu, cpu, cpu, cpu),
             lambda: m.mla_gather_cache_scaled(cpu, cpu, cpu, cpu, cpu, 0),
             lambda: m.mla_prefill_attn_window(cpu, cpu, cpu, cpu, cpu, 1, window=1, sm_scale=1.0)):
    try:
        call()
    except {error} as e:
        assert "{text}" in str(e), e
    else:
        raise AssertionError("no {error}")
"""

# the loader looks whether the file is there
MISSING = """
real = os.path.exists
os.path.exists = lambda p: not str(p).endswith("_mla_binding.so") and real(p)
"""


def _run(**kw):
    r = subprocess.run([sys.executable, "-c", CODE.format(**kw)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_without_the_compiled_module():
    _run(before=MISSING, error="ImportError", text="_mla_binding.so is missing")


def test_with_it():
    _run(before="", error="ValueError", text="must be a CUDA tensor")
