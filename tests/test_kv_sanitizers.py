"""The key/value cache's host code under AddressSanitizer and
UndefinedBehaviorSanitizer: csrc/kv_api.hip and csrc/api.hip compiled as host
C++ with launch stubs in place of the kernel files, and the cache's CPU tests
rerun on that build in a child interpreter.  Any report fails the run.  No
GPU."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantization_error_compensation_amd", "csrc")
OUT = os.path.join(ROOT, "tests", "_build")
SAN = ["-fsanitize=address,undefined", "-fno-omit-frame-pointer", "-fno-sanitize-recover=all", "-g",
       "-O1"]


def test_cache_host_code_is_clean_under_asan_and_ubsan():
    os.makedirs(OUT, exist_ok=True)
    so = os.path.join(OUT, "libspear_ec_kv_host_san.so")
    stubs = [os.path.join(ROOT, "tests", f) for f in ("sanitize_stubs.cpp", "kv_sanitize_stubs.cpp")]
    subprocess.check_call(
        ["g++", "-std=c++17", "-shared", "-fPIC", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-x", "c++", os.path.join(CSRC, "api.hip"),
         os.path.join(CSRC, "kv_api.hip"), os.path.join(CSRC, "scheduler.cpp"), *stubs, "-x", "none",
         "-L/opt/rocm/lib", "-Wl,-rpath,/opt/rocm/lib", "-lamdhip64", "-o", so])
    asan = subprocess.check_output(["gcc", "-print-file-name=libasan.so"], text=True).strip()
    env = dict(os.environ, LD_PRELOAD=asan, SPEAR_EC_LIB=so,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([sys.executable, "-m", "pytest", "tests/test_kv_host.py", "-q", "-x", "-p",
                          "no:cacheprovider"], cwd=ROOT, env=env, capture_output=True, text=True,
                         timeout=900)
    out = res.stdout + res.stderr
    assert res.returncode == 0, out[-4000:]
    for marker in ("AddressSanitizer", "runtime error:", "LeakSanitizer"):
        assert marker not in out, out[-4000:]
    assert " passed" in out
