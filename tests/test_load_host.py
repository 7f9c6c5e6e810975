"""Loading the library and reading its constants needs no torch (no GPU)."""

import os
import subprocess
import sys

from nsa_block_selection_gb300 import _lib
from nsa_block_selection_gb300.build import ROOT

SCRIPT = """
import sys
sys.modules["torch"] = None  # an import of it fails
import nsa_block_selection_gb300 as nsa
from nsa_block_selection_gb300 import _lib
assert nsa.load().nsa_version() >= 100
assert nsa.status_string(0)
assert _lib.norm_rope_bwd_workspace_bytes(1, 8, 64) > 0
assert _lib.swa_bwd_workspace_bytes(1, 8, 8, 2, 1, 64) > 0
assert _lib.bwd_workspace_bytes(1, 64, 64, 8, 1, 64, 2, 32) > 0
print("loaded")
"""


def test_load_without_torch():
    if not os.path.exists(_lib.LIB_PATH):
        from nsa_block_selection_gb300.build import build

        build()
    run = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
    assert run.stdout.strip() == "loaded"


def test_load_before_torch():
    """The calls that take torch's tensors bind it themselves, whenever the
    library was loaded."""
    script = ("from nsa_block_selection_gb300 import _lib, load; load()\n"
              "import torch\n"
              "q, k = torch.zeros(1, 8, 4, 64).bfloat16(), torch.zeros(1, 8, 2, 64).bfloat16()\n"
              "lse = torch.zeros(1, 4, 8)\n"
              "for call in (lambda: _lib.swa_bwd(q, k, k, q, lse, q), lambda: _lib.qk_norm_rope(q, k),\n"
              "             lambda: _lib.qk_norm_rope_bwd(q, k, q, k)):\n"
              "    try:\n"
              "        call()\n"
              "    except ValueError as e:\n"
              "        assert 'CUDA' in str(e), e\n"
              "    else:\n"
              "        raise AssertionError('taken')\n"
              "print('refused')\n")
    run = subprocess.run([sys.executable, "-c", script], cwd=ROOT, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
    assert run.stdout.strip() == "refused"
