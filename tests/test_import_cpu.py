"""What importing the package costs: no torch until an operator is used."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


@pytest.mark.parametrize("module", ["gaussian_splatting_raster_b200",
                                    "gaussian_splatting_raster_b200.build",
                                    "gaussian_splatting_raster_b200.runner"])
def test_import_leaves_torch_out(module):
    """Building and loading the library, and planning with the package's constants, need no torch."""
    r = _run(f"import sys; sys.modules['torch'] = None\nimport {module}")
    assert r.returncode == 0, r.stderr


def test_operators_are_public():
    r = _run("import gaussian_splatting_raster_b200 as P\n"
             "from gaussian_splatting_raster_b200 import *\n"
             "assert all(callable(getattr(P, n)) for n in "
             "('lookup', 'lookup_backward', 'ffn', 'ffn_backward', 'rows_status'))\n"
             "assert P.ffn is ffn and P.rows.ffn is ffn\n"
             "try:\n    P.nothing\nexcept AttributeError as e:\n    assert 'nothing' in str(e)\n"
             "else:\n    raise SystemExit(1)")
    assert r.returncode == 0, r.stderr


def test_the_operators_module_is_an_attribute():
    r = _run("import gaussian_splatting_raster_b200 as P\nassert P.rows.lookup is P.lookup")
    assert r.returncode == 0, r.stderr
