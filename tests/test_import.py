"""What importing the package says where its extension module is missing, broken or built against another torch."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BEFORE = {
    "another torch": "import torch; torch.__version__ = type(torch.__version__)('9.9.0')",
    "missing": "import sys; sys.modules['fine_grained_blockwise_amd._tensors'] = None",
    "an earlier source": "import sys, types; sys.modules['fine_grained_blockwise_amd._tensors'] = "
                         "types.ModuleType('fine_grained_blockwise_amd._tensors')",
}


@pytest.mark.parametrize("case", sorted(BEFORE))
def test_import_says_what_to_do(case):
    code = BEFORE[case] + """
try:
    import fine_grained_blockwise_amd
except ImportError as e:
    print("ImportError:", e)
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert "ImportError:" in r.stdout and "_tensors" in r.stdout and "build()" in r.stdout, r.stdout + r.stderr[-500:]
    if case == "another torch":
        assert "9.9.0" in r.stdout


def test_the_module_is_this_python_s_and_torch_s():
    import sysconfig

    import torch

    import fine_grained_blockwise_amd as fgb
    assert fgb._tensors.torch_version == torch.__version__
    assert fgb._tensors.__file__.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
