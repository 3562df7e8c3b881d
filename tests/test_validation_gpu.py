"""MGEMM_VALIDATE=1 in the fp8 products, the row quantizers and the combine's
gradient.  The library reads the variable once per process, so the calls run in
a child (gpu_validate_child.py)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu


def test_validation_of_offsets_and_of_rows_named_twice():
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, MGEMM_VALIDATE="1", PYTHONPATH=os.pathsep.join([os.path.dirname(here), here, os.environ.get("PYTHONPATH", "")]))
    print("[case] child with MGEMM_VALIDATE=1", flush=True)
    p = subprocess.run([sys.executable, "-u", os.path.join(here, "gpu_validate_child.py")], env=env, capture_output=True, text=True, timeout=100)
    print(p.stdout[-3000:], p.stderr[-3000:], flush=True)
    assert p.returncode == 0 and p.stdout.count("[child] refused") == 13 and "[child] ok" in p.stdout
