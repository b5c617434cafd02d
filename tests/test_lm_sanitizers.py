"""AddressSanitizer + UndefinedBehaviorSanitizer on the argument checks of the
embedding, cross-entropy and gradient-list entry points (lm_api.cpp on host stubs).
CPU only; any report aborts the program."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "bit_microscaled_numerics_amd", "csrc")


def test_argument_checks_under_sanitizers(tmp_path):
    exe = str(tmp_path / "lm_api_asan")
    subprocess.run(["g++", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-g", "-O1",
                    "-std=c++17", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", f"-I{CSRC}",
                    f"-I{os.path.join(ROOT, 'include')}",
                    os.path.join(HERE, "sanitize", "lm_api_driver.cpp"),
                    os.path.join(HERE, "sanitize", "lm_api_stubs.cpp"),
                    os.path.join(CSRC, "lm_api.cpp"), "-o", exe], check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], env=env, capture_output=True, text=True)
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-2000:])
    assert "unexpected statuses: 0" in r.stdout
