"""The launches of the training operators, on the host: the launchers of
norm.hip, route.hip and distill.hip and the C entry points under the host
sanitizers, with a HIP runtime that records launches
(tests/host_fake/launch_driver.cpp)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "ring_allreduce_rs_amd", "csrc")
FAKE = os.path.join(ROOT, "tests", "host_fake")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/llvm/bin/clang++"
SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
       "-Xarch_host", "-fno-sanitize-recover=all"]

pytestmark = pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)),
                                reason="needs the ROCm toolchain")


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("launches")
    common = ["-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-x", "hip",
              "--cuda-host-only", f"-I{ROOT}/include", f"-I{CSRC}", f"-I{FAKE}"] + SAN
    objs = []
    for src in (*(os.path.join(CSRC, f) for f in ("norm.hip", "route.hip", "distill.hip",
                                                  "ops_api.cpp", "ar_api.cpp", "dispatch.hip")),
                os.path.join(FAKE, "fake_hip.cpp"), os.path.join(FAKE, "launch_driver.cpp")):
        obj = str(tmp / (os.path.basename(src) + ".o"))
        r = subprocess.run([HIPCC] + common + ["-c", src, "-o", obj],
                           capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, f"compile {src}:\n{r.stderr[-4000:]}"
        objs.append(obj)
    exe = str(tmp / "launch_driver")
    # (the device code that the host objects name is not there and not asked for)
    r = subprocess.run([CLANG, "-fsanitize=address,undefined", "-no-pie",
                        "-Wl,--unresolved-symbols=ignore-all", "-o", exe] + objs,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, f"link:\n{r.stderr[-4000:]}"

    def run(section):
        r = subprocess.run([exe, section], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and "ALL OK" in r.stdout, (r.stdout + r.stderr)[-6000:]
    return run


def test_more_rows_than_blocks(driver):
    driver("rows")


def test_the_widest_rows(driver):
    driver("widths")


def test_temperatures_whose_inverse_overflows(driver):
    driver("temperatures")


def test_scratch_holds_what_the_kernels_leave(driver):
    driver("scratch")
