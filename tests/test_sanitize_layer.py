"""The host ABI of the operators between the projections (wq_layer_abi.cpp)
under AddressSanitizer and UndefinedBehaviorSanitizer, with stub launchers (CPU
only; tests/c/layer_abi_sanitize.cpp)."""
import os

from tests.test_sanitize_host import CSRC, ROOT, SAN, _env, _run, tmp  # noqa: F401  (tmp is a fixture)


def test_layer_abi_under_sanitizers(tmp):  # noqa: F811
    exe = os.path.join(tmp, "layer_abi_sanitize")
    rc, out = _run(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + os.path.join(ROOT, "include"), os.path.join(CSRC, "wq_layer_abi.cpp"),
                    os.path.join(ROOT, "tests", "c", "layer_abi_sanitize.cpp"),
                    "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe], None, 300)
    assert rc == 0, out
    rc, out = _run([exe], _env(tmp), 300)
    assert rc == 0 and "all checks passed" in out and "runtime error" not in out, out
