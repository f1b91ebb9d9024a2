"""Host code of linear attention, window attention and the norms of queries and keys under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): ``sanitize/mixer_checks.c`` with their sources, sanitizers on the host pass."""
import os
import subprocess

import pytest

# (left out of copies of the tree that only run GPU tests)
san = pytest.importorskip("tests.test_sanitizers")
CLANG, CSRC, ENV, HIP_SAN, HIPCC, ROOT, SAN = san.CLANG, san.CSRC, san.ENV, san.HIP_SAN, san.HIPCC, san.ROOT, san.SAN
_need, _run = san._need, san._run

SOURCES = ["mamba_linear.hip", "mamba_linear_bwd.hip", "mamba_window.hip", "mamba_window_bwd.hip", "mamba_window_step.hip",
           "mamba_qk_norm.hip"]


def test_c_abi_of_the_mixers_under_asan_ubsan(tmp_path):
    _need(HIPCC)
    _need(CLANG)
    include = ["-I", os.path.join(ROOT, "include")]
    procs = []
    for f in SOURCES:
        obj = str(tmp_path / (f + ".o"))
        procs.append((obj, subprocess.Popen([HIPCC] + HIP_SAN + include + ["-c", os.path.join(CSRC, f), "-o", obj],
                                            stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)))
    objs = []
    for obj, p in procs:
        _, err = p.communicate(timeout=600)
        assert p.returncode == 0, err
        objs.append(obj)
    drv = str(tmp_path / "mixer_checks.o")
    r = _run([CLANG, "-O1", "-g", "-std=c11", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
              "-fno-sanitize-recover=all"] + include + ["-c", os.path.join(SAN, "mixer_checks.c"), "-o", drv])
    assert r.returncode == 0, r.stderr
    exe = str(tmp_path / "mixer_checks")
    r = _run([HIPCC, "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-o", exe, drv] + objs)
    assert r.returncode == 0, r.stderr
    # the HIP runtime keeps allocations until exit; leak reports would be its own
    r = _run([exe], env=dict(ENV, ASAN_OPTIONS="detect_leaks=0"))
    assert r.returncode == 0 and "clean" in r.stdout, r.stdout + r.stderr
