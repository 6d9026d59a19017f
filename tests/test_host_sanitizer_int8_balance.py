"""The host code of the 8-bit integer, norm and balance-loss calls under AddressSanitizer and
UndefinedBehaviorSanitizer: the library built as in test_host_sanitizer, with
``tests/host_sanitizer_int8_balance.c``, over the extremes of the sizes."""
import os
from concurrent.futures import ThreadPoolExecutor

import pytest

import test_host_sanitizer as hs
from moe_expert_layer_segment_amd import build


@pytest.mark.skipif(not os.path.exists(hs.CLANG) or not os.path.exists(build.hipcc()),
                    reason="ROCm clang / hipcc not available")
def test_host_code_of_int8_and_balance_calls(tmp_path):
    flags = [f for f in build.common_flags() if f != "-O3"] + ["-O1", "-g"] + hs.SAN

    def compile_one(src):
        out = str(tmp_path / (os.path.splitext(src)[0] + ".o"))
        lang = ["-x", "hip"] if src.endswith(".cpp") else []
        hs._run([build.hipcc()] + lang + flags + ["-c", os.path.join(build.CSRC, src), "-o", out])
        return out

    with ThreadPoolExecutor(max_workers=min(8, len(build.SOURCES))) as ex:
        objs = list(ex.map(compile_one, build.SOURCES))
    drv, exe = str(tmp_path / "driver.o"), str(tmp_path / "driver")
    hs._run([hs.CLANG, "-O1", "-g", "-I", build.INCLUDE, "-c",
             os.path.join(hs.ROOT, "tests", "host_sanitizer_int8_balance.c"), "-o", drv])
    hs._run([hs.CLANG + "++", "-fsanitize=address,undefined", drv] + objs +
            ["-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1")
    res = hs.subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "all host checks passed" in res.stdout
