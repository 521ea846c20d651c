"""The argument checks of the operators around the products under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU): tests/sanitize/block_driver.cpp."""
import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.join(HERE, "sanitize"))


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc") or shutil.which("gcc") is None, reason="hipcc not available")
def test_block_checks_under_sanitizers(tmp_path):
    import build as sb
    host = [f for s in sb.SAN for f in ("-Xarch_host", f"-fsanitize={s}")]
    common = ["-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "--offload-arch=gfx950", "-Xarch_host",
              "-fno-sanitize-recover=all", *host, "-I", sb.CSRC]
    objs = []
    for src, extra in ((os.path.join(sb.CSRC, "api.hip"), []),
                       (os.path.join(sb.CSRC, "block_api.hip"), ["--cuda-host-only"]),
                       (os.path.join(HERE, "sanitize", "block_driver.cpp"), ["--cuda-host-only"])):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        sb._run([os.path.join(sb.ROCM, "bin", "hipcc"), *common, *extra, "-x", "hip", "-c", src, "-o", obj])
        objs.append(obj)
    exe = str(tmp_path / "block_driver")
    lib = os.path.join(sb.ROCM, "lib")
    sb._run([os.path.join(sb.ROCM, "llvm", "bin", "clang++"), *[f"-fsanitize={s}" for s in sb.SAN], "-o", exe, *objs,
             "-L", lib, "-lamdhip64", f"-Wl,-rpath,{lib}"])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("OK"), r.stdout + r.stderr
