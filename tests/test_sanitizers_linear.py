"""The C-ABI layer of linear attention and layer norm under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): a host-only library of gdn_api.cpp and gdn_linear_api.cpp
with launchers that report no device, and the C-ABI tests run against it in a child process."""
import os
import subprocess

import test_sanitizers as san

pytestmark = san.pytestmark


def test_linear_abi_under_asan_ubsan(tmp_path):
    lib_oracle, lib_gdn = str(tmp_path / "liboracle_san.so"), str(tmp_path / "libgdn_san.so")
    san._build_oracle(os.path.join(san.ROOT, "oracle", "gdn_oracle.c"), lib_oracle)
    sources = [os.path.join(san.CSRC, "gdn_api.cpp"), os.path.join(san.CSRC, "gdn_linear_api.cpp"),
               os.path.join(san.HERE, "sanitize", "stub_launch.cpp"),
               os.path.join(san.HERE, "sanitize", "stub_launch_linear.cpp")]
    subprocess.run(["g++", *san.SAN, "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    f"-I{os.path.join(san.ROOT, 'include')}", f"-I{san.CSRC}", "-o", lib_gdn, *sources,
                    "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"], check=True)
    r = san._run_child(lib_oracle, lib_gdn, ["test_linear_abi.py"])
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-40:])
    assert r.returncode == 0, tail
    assert "passed" in r.stdout and "ERROR: AddressSanitizer" not in r.stderr, tail
    assert "runtime error" not in r.stderr, tail
