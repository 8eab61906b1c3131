"""When the binding maps its compiled parts: not before lib(), so that a process which imports the
package, builds it and then uses it runs what it built."""
import subprocess
import sys

from conftest import ROOT

CODE = """
import block_scaled_precision_act_b200 as bsp
def mapped(name):
    return any(name in line for line in open("/proc/self/maps"))
import block_scaled_precision_act_b200.nn
import block_scaled_precision_act_b200.build
assert not mapped("libbsp.so") and not mapped("_fastcall.so") and bsp._fastcall is None
bsp.lib()
assert mapped("libbsp.so") and mapped("_fastcall.so")
assert bsp._fastcall.gemv and bsp._fastcall.append and bsp._fastcall.attention
"""


def test_nothing_is_mapped_on_import():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
