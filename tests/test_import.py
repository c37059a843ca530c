"""Importing the package (no GPU needed)."""
import subprocess
import sys

from conftest import ROOT


def _python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, check=True).stdout.split()


def test_the_package_does_not_import_torch():
    """Users of the step alone (plain addresses, numpy arrays) do not pay for it."""
    assert _python("import sys, random_gradient_projection_b200 as p; print('torch' in sys.modules, hasattr(p, 'grape'))") == [
        "False", "True"]


def test_the_language_model_entry_points_come_with_the_package():
    code = "import random_gradient_projection_b200 as p; print(p.lm.__name__, hasattr(p, 'no_such_module')); "
    code += "from random_gradient_projection_b200 import lm; print(lm is p.lm)"
    assert _python(code) == ["random_gradient_projection_b200.lm", "False", "True"]
