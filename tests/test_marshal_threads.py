"""Other Python threads run while a call is inside an entry point (CPU).

The entry point is a stand-in: a library loaded first, whose symbol the native module binds to.  It waits, for a few
seconds at most, until another Python thread has told it to go on.
"""
import subprocess
import sys

STUB = """
#include <unistd.h>
volatile int entered = 0, go = 0;
int mamba_gated_norm_fwd() {
  entered = 1;
  for (int i = 0; i < 5000 && !go; ++i) usleep(1000);
  return go ? 0 : 77;
}
"""
CODE = """
import ctypes, os, sys, threading, time
stub = ctypes.CDLL(sys.argv[1], mode=os.RTLD_GLOBAL | os.RTLD_NOW)
import torch
from selective_state_space_47_amd import binding
m = binding._marshal()
entered, go = (ctypes.c_int.in_dll(stub, n) for n in ("entered", "go"))
status = []
t = threading.Thread(target=lambda: status.append(m.call(binding._GATED_FWD, 0, 0, 1.0, 0, None, None, None, None)))
t.start()
while not entered.value and t.is_alive():
    time.sleep(0.001)
go.value = 1
t.join()
print(entered.value, status)
"""


def test_other_threads_run_during_a_call(tmp_path):
    src, lib = tmp_path / "stub.c", tmp_path / "stub.so"
    src.write_text(STUB)
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-w", "-o", str(lib), str(src)], check=True)
    r = subprocess.run([sys.executable, "-c", CODE, str(lib)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split("\n")[0] == "1 [0]", r.stdout
