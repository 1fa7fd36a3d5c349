"""The host-side tests call the C functions with made-up addresses, which are never looked at as long as no call gets past its
argument checks to a device. Where there is no GPU one that does ends in QG_ERR_CUDA; where there is one it must not be made.
Here a child process without devices runs those tests as if there were one, and counts the calls that would have launched."""
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))

CHILD = r'''
import sys
import pytest
sys.path[:0] = [ROOT, ROOT + "/tests"]
import gemm_q4_q8_gb300 as qg
from gemm_q4_q8_gb300 import build
build.build()
lib, past = qg.load(), []

def counted(name, f):
    def call(*a):
        st = f(*a)
        if st == qg.QG_ERR_CUDA:
            past.append(name)
        return st
    return call

for n in qg.EXPORTS:
    f = getattr(lib, n)
    if getattr(f, "restype", None) is not None and n not in ("qg_device_error", "qg_status_str"):
        w = counted(n, f)
        w.argtypes, w.restype = f.argtypes, f.restype
        setattr(lib, n, w)

class AsIf:
    ran = 0
    def pytest_collection_finish(self, session):
        import conftest
        conftest.gpu_available = lambda: True
    def pytest_runtest_logreport(self, report):
        AsIf.ran += report.when == "call" and report.passed

rc = pytest.main([ROOT + "/tests/" + FILE, "-q", "-m", "not gpu", "-p", "no:cacheprovider"], plugins=[AsIf()])
print("RAN", AsIf.ran, "RC", int(rc), "PAST", past)
'''


@pytest.mark.parametrize("file", ["test_abi.py", "test_attn_abi.py", "test_binding_threads.py", "test_rope_plan.py"])
def test_no_call_gets_to_the_device(file):
    code = f"ROOT, FILE = {os.path.dirname(HERE)!r}, {file!r}\n" + CHILD
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, CUDA_VISIBLE_DEVICES=""), capture_output=True,
                       text=True, timeout=600)
    last = r.stdout.strip().splitlines()[-1]
    assert last.endswith("PAST []") and " RC 0 " in last and not last.startswith("RAN 0 "), r.stdout[-2000:] + r.stderr[-2000:]
