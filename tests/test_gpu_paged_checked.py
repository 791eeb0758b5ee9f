"""The paged calls under the range-checked build (libeta_checked.so): their tests pass
unchanged without a range report, and a group whose rows do not hold the same prefix is
reported."""
import os
import subprocess
import sys

import pytest

from test_gpu_checked import REPORT, ROOT, _checked_env

pytestmark = pytest.mark.gpu


def _run(args):
    env = _checked_env()
    env["PYTHONPATH"] = os.pathsep.join((ROOT, os.path.join(ROOT, "tests")))
    p = subprocess.run([sys.executable, *args], env=env, capture_output=True, text=True,
                       timeout=1500, cwd=ROOT)
    tail = "\n".join((p.stdout + p.stderr).splitlines()[-30:])
    assert p.returncode == 0, tail
    assert REPORT not in p.stdout and REPORT not in p.stderr, tail
    return p.stdout


def test_paged_suites_pass_under_the_checked_build():
    out = _run(["-m", "pytest", "-x", "-q", "-s", "-m", "gpu", "-p", "no:cacheprovider",
                "tests/test_gpu_pages.py", "tests/test_gpu_paged_decode.py",
                "tests/test_gpu_shared_decode.py", "tests/test_gpu_paged_edges.py"])
    assert " passed" in out


def test_a_prefix_that_rows_do_not_share_is_reported():
    out = _run(["-c", """
import torch
from long_context_decoding_eta_b200 import _lib as L
from long_context_decoding_eta_b200.paged import PagedEtaDecoder
from test_gpu_shared_decode import shared_cache
assert L.eta_build_checked()
c, off, pre = shared_cache([(40, [40 * 64 + 9] * 5), (2, [130, 128, 100, 140])], 2, 64, 64)
dec = PagedEtaDecoder(c, 4, T=None)
q = torch.randn(9, 4, 64).to(torch.bfloat16).cuda()

def status():
    dec.shared_decode(q, off, pre)
    torch.cuda.synchronize()
    s = int(dec.dev_status)
    dec.dev_status.zero_()
    return s

print("same", status())
for row, j in ((3, 39), (4, 0), (8, 1)):
    page = int(c.table[row, j])
    c.table[row, j] = int(c.table[row, -1]) if row < 5 else int(c.table[0, 0])
    print("other", status())
    c.table[row, j] = page
c.table[7, 0] = int(c.table[0, 0])       # shorter than the prefix: read by itself
print("same", status())
"""])
    assert out.split() == ["same", "0"] + ["other", "64"] * 3 + ["same", "0"]
