"""The argument validation of the operators around the selection under AddressSanitizer and
UndefinedBehaviorSanitizer, as test_host_sanitize.py does it for the selection: the driver in
host_sanitize/operators_validation.cpp calls each of their entry points with sizes, strides, positions and
pointers at the ends of their types, and none of its calls gets as far as a HIP call."""
import concurrent.futures as cf
import glob
import os
import subprocess

import pytest

from exact_top_token_amd import build as hkbuild

base = pytest.importorskip("test_host_sanitize")


def _older(obj, sources):
    return not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(s) for s in sources)


@pytest.mark.timeout(600)
def test_operators_validation_under_host_sanitizers():
    os.makedirs(base.OUT, exist_ok=True)
    cc = hkbuild.hipcc()
    sources = glob.glob(os.path.join(hkbuild.CSRC, "*")) + glob.glob(os.path.join(hkbuild.INCLUDE, "*"))
    jobs, objs = [], []
    for src in hkbuild.SOURCES:  # the other test's objects where they are up to date
        obj = os.path.join(base.OUT, src.replace(".hip", ".o"))
        objs.append(obj)
        if _older(obj, sources):
            jobs.append([cc, *hkbuild.FLAGS, *base.SAN, "-O1", "-g", "-c", os.path.join(hkbuild.CSRC, src), "-o", obj])
    with cf.ThreadPoolExecutor(8) as ex:
        list(ex.map(base._compile, jobs))
    drv = os.path.join(base.OUT, "operators_validation.o")
    base._compile([cc, "-x", "c++", *base.SAN, "-g", "-I", hkbuild.INCLUDE, "-c",
                   os.path.join(base.HERE, "host_sanitize", "operators_validation.cpp"), "-o", drv])
    exe = os.path.join(base.OUT, "operators_validation")
    base._compile([cc, f"--offload-arch={hkbuild.ARCH}", *base.SAN, drv, *objs, "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    p = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, env=env, timeout=120)
    print(p.stdout[-4000:])
    assert p.returncode == 0, p.stdout[-4000:]
    assert "ok: 0 failure(s)" in p.stdout
