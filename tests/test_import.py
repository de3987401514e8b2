"""Importing the package, also by ``import *``, needs neither torch nor a built library; the
serving operators are there all the same."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _python(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("block", ["", "sys.modules['torch'] = None; "])
def test_star_import_loads_no_torch(block):
    _python("import sys; " + block + "had = set(sys.modules); "
            "from gated_delta_rule_62_amd import *; "
            "assert sys.modules.get('torch') is None; "
            "assert 'gated_delta_rule_62_amd.serving' not in sys.modules; "
            "assert kda_fwd.__name__ == 'kda_fwd' and kda_step.__name__ == 'kda_step'")


def test_star_import_without_the_compiled_calls():
    _python("import torch, gated_delta_rule_62_amd as kda\n"
            "kda.CALLS_PATH = kda.CALLS_PATH + '.missing'\n"
            "import sys; sys.modules['gated_delta_rule_62_amd._serving_calls'] = None\n"
            "from gated_delta_rule_62_amd import *\n"
            "try:\n    kda_step()\n"
            "except ImportError as e:\n    assert 'not built' in str(e), e\n"
            "else:\n    raise AssertionError('called')\n")


def test_a_name_taken_early_calls_the_operator():
    _python("import sys\nfrom gated_delta_rule_62_amd import kda_la_workspace_bytes as early\n"
            "assert 'torch' not in sys.modules\n"
            "assert early(200, 2, 4, 128, segment=64) == (200 // 64 + 3) * 4 * (128 * 128 + 1) * 4\n"
            "import gated_delta_rule_62_amd as kda\n"
            "from gated_delta_rule_62_amd import serving\n"
            "assert kda.kda_la_workspace_bytes is serving.kda_la_workspace_bytes\n"
            "assert kda.kda_step is serving.kda_step\n")


def test_names_are_the_functions_themselves_beside_torch():
    _python("import torch\nfrom gated_delta_rule_62_amd import kda_step\n"
            "from gated_delta_rule_62_amd import serving\nassert kda_step is serving.kda_step\n")
