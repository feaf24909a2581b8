"""The host code of the operators around the experts (abi_block.cpp, with abi.cpp) under AddressSanitizer and
UndefinedBehaviorSanitizer, as test_abi_sanitize.py does for abi.cpp alone."""
import os
import subprocess
import sys

from test_abi_sanitize import ROOT, OUT, sanitized_lib  # noqa: F401  (the fixture)

BOTH = os.path.join(os.path.dirname(OUT), "libw4a8moe_block_sanitize.so")


def test_block_checks_under_sanitizers(sanitized_lib):  # noqa: F811
    csrc = f"{ROOT}/quantized_grouped_gemm_token_amd/csrc"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fPIC", "-shared", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           f"-I{ROOT}/include", f"-I{csrc}", f"{csrc}/abi.cpp", f"{csrc}/abi_block.cpp",
           f"{ROOT}/tests/sanitize/launch_stubs.cpp", f"{ROOT}/tests/sanitize/block_stubs.cpp",
           "-L/opt/rocm/lib", "-Wl,-rpath,/opt/rocm/lib", "-lamdhip64", "-o", BOTH]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-s", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_block_cpu.py")],
                       env=dict(sanitized_lib, W4A8_MOE_LIB=BOTH), capture_output=True, text=True, cwd=ROOT,
                       timeout=300)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0, tail
    assert "AddressSanitizer" not in tail and "runtime error" not in tail, tail
    nm = subprocess.run(["nm", "-C", BOTH], capture_output=True, text=True, check=True).stdout.splitlines()
    ours = [line.split(maxsplit=2) if line[0] != " " else ["", *line.split(maxsplit=1)] for line in nm
            if "w4a8::" in line]
    assert any("launch_norm" in name for _, _, name in ours)
    assert not [name for _, kind, name in ours if kind in "wU"]
