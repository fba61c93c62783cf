"""The debug build against the release build over the kernels of the FP8
layer, the layer norm and the distillation loss (tests/tail_debug_workload.py):
no range check fails, every output is bit-identical."""
from __future__ import annotations

import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.join(os.path.dirname(HERE), "bit_nf4_quantized_21_b200")


def _run(lib: str) -> dict:
    r = subprocess.run([sys.executable, os.path.join(HERE, "tail_debug_workload.py")], env=dict(os.environ, QLORA_LIB=lib),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


def test_debug_build_checks_pass_and_match_release():
    dbg, rel = (_run(os.path.join(PKG, n)) for n in ("libqlora_debug.so", "libqlora.so"))
    assert dbg.pop("checks") == 1 and rel.pop("checks") == 0
    assert dbg.pop("range_site") == 0 and rel.pop("range_site") == 0
    diff = [k for k in rel if rel[k] != dbg.get(k)]
    assert not diff, f"outputs differ between the debug and release builds: {diff}"
