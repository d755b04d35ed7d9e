"""CPU: the host side of the quantized cache's and the pages' entry points
(argument checks, size arithmetic, plans and dispatch) under the address and
undefined-behaviour sanitizers.

cache_api.hip and the three sources with its launchers are compiled with both
sanitizers on their host side only and linked with the library's other objects
as built; tests/test_cache_abi.py then runs through the Python
binding against that build, none of it reaching the GPU.  Undefined behaviour
aborts (no recovery), so any report fails the test."""

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

from gemm_lora_shrink_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "gemm_lora_shrink_amd")
CHECKED = ("cache_api", "quantized", "pages", "attend_quantized")
SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
       "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer"]

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc is not available")


def _run(cmd, **kw):
    res = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert res.returncode == 0, f"{' '.join(cmd[:3])} ... failed:\n{res.stdout[-3000:]}\n{res.stderr[-3000:]}"
    return res


def test_cache_binding_checks_under_sanitizers(tmp_path):
    rt = subprocess.run(["hipcc", "-print-file-name=libclang_rt.asan-x86_64.so"], capture_output=True,
                        text=True).stdout.strip()
    if not rt or not os.path.exists(rt):
        pytest.skip("the sanitizer runtime is not installed")
    names = [s[:-len(".hip")] for s in build.SOURCES]
    others = [os.path.join(PKG, "_build", f"{n}.o") for n in names if n not in CHECKED]
    if not all(os.path.exists(o) for o in others):
        pytest.skip("the library has not been built")
    lib = str(tmp_path / "liblora_san.so")

    def compiled(name):
        o = str(tmp_path / f"{name}.o")
        _run(["hipcc", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-fvisibility=hidden",
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", *SAN, "-I", os.path.join(ROOT, "include"),
              "-c", os.path.join(PKG, "csrc", f"{name}.hip"), "-o", o])
        return o

    with ThreadPoolExecutor(len(CHECKED)) as pool:
        checked = list(pool.map(compiled, CHECKED))
    _run(["hipcc", "--offload-arch=gfx950", "-shared", "-fPIC", *SAN, "-o", lib, *checked, *others])
    env = dict(os.environ, LD_PRELOAD=rt, LORA_MI355X_LIB=lib,
               ASAN_OPTIONS="detect_leaks=0:verify_asan_link_order=0:detect_odr_violation=0")
    probe = _run([sys.executable, "-c", "import gemm_lora_shrink_amd as g; g._load(); "
                  "print(sum('liblora_san' in l for l in open('/proc/self/maps')))"], env=env, cwd=ROOT, timeout=300)
    assert int(probe.stdout.split()[-1]) > 0, "the sanitized build was not the one loaded"
    res = _run([sys.executable, "-m", "pytest", os.path.join(ROOT, "tests", "test_cache_abi.py"), "-q", "-x",
                "-m", "not gpu", "-p", "no:cacheprovider"], env=env, cwd=ROOT, timeout=600)
    assert " passed" in res.stdout
    assert "AddressSanitizer" not in res.stderr and "runtime error" not in res.stderr + res.stdout
