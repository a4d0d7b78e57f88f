"""On the CPU: the sizes and lines that the GPU tests run the experts' products at
(tests/product_cases.py) take the kernels that they are said to, and no call
takes another (tests/host_fake/product_plan_driver.cpp runs the launcher)."""

import os
import re
import shutil
import subprocess

import pytest

from tests import product_cases as pc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "ring_allreduce_rs_amd", "csrc")
FAKE = os.path.join(ROOT, "tests", "host_fake")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/llvm/bin/clang++"
SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
       "-Xarch_host", "-fno-sanitize-recover=all"]
KINDS = ("out", "drows", "dweights")

pytestmark = pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)),
                                reason="needs the ROCm toolchain")


@pytest.fixture(scope="module")
def launched(tmp_path_factory):
    """calls -> the kernel of each, as product_cases.kernel names it."""
    tmp = tmp_path_factory.mktemp("plan")
    common = ["-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-x", "hip",
              "--cuda-host-only", f"-I{ROOT}/include", f"-I{CSRC}", f"-I{FAKE}"] + SAN
    objs = []
    for src in (*(os.path.join(CSRC, f) for f in ("ar_api.cpp", "model_api.cpp", "dispatch.hip",
                                                  "product.hip")),
                *(os.path.join(FAKE, f) for f in ("fake_hip.cpp", "product_plan_driver.cpp"))):
        obj = str(tmp / (os.path.basename(src) + ".o"))
        r = subprocess.run([HIPCC] + common + ["-c", src, "-o", obj],
                           capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, f"compile {src}:\n{r.stderr[-4000:]}"
        objs.append(obj)
    exe = str(tmp / "driver")
    # (the launchers and device code that the objects name beside are not asked for)
    r = subprocess.run([CLANG, "-fsanitize=address,undefined", "-no-pie",
                        "-Wl,--unresolved-symbols=ignore-all", "-o", exe] + objs,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, f"link:\n{r.stderr[-4000:]}"

    def run(calls):
        text = "".join(" ".join(map(str, c)) + "\n" for c in calls)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=300)
        lines = r.stdout.split("\n")
        assert r.returncode == 0 and lines[-2:] == ["ALL OK", ""], r.stderr[-4000:]
        return [kernel(line) for line in lines[:-2]]
    return run


def kernel(line):
    first, *more = line.split(";")[:-1]
    m = re.search(r"k_product<(\d), .*ProductKind\)(\d), (true|false), (true|false), "
                  r".*Shape<(\d+), (\d+), ", first)
    assert m and all("k_product_join" in k for k in more), line
    return KINDS[int(m[2])], int(m[1]), m[3][0] + m[4][0], f"{m[5]}x{m[6]}", bool(more)


def call(kind, eb, rows, experts, hidden, out, lines):
    sa, ea, sb, eb_ = lines
    wa, wb = pc.widths(kind, hidden, out)
    return (KINDS.index(kind), 2 if eb == 2 else 1, rows, experts, hidden, out, wa + ea,
            wb + eb_ if wb else 0, sa, sb)


def test_cases_take_the_kernels_that_they_name(launched):
    cases = pc.cases()
    for c, got in zip(cases, launched([call(*sizes, lines) for sizes, lines in cases])):
        assert got == pc.kernel(*c), c


def test_no_call_takes_another(launched):
    named = {pc.kernel(*c) for c in pc.cases()}
    widths = (1, 7, 24, 64, 72, 130, 264, 520, 771, 1001, 2048, 2056, 4104, 8200, 16392, 1 << 20)
    calls = [call(k, eb, n, e, h, o, lines)
             for k in KINDS for eb in (2, 4)
             for n in (1, 5, 40, 130, 300, 520, 1100, 4100, 16400, 66000, 1000003)
             for e in (1, 3, 7, 26, 64, 256, 1024) for h in widths for o in widths
             for lines in (((0, 0, 0, 0), (1, 0, 1, 0)) if eb == 2 else ((0, 0, 0, 0),))
             if max(n * h, n * o, e * h * o) < 10 ** 11]
    found = set(launched(calls))
    assert len(found) > 40 and found <= named, found - named


def test_groups_add_up():
    for kind, eb, n, experts, hidden, out in pc.SHAPES:
        g = pc.groups(n, experts)
        assert len(g) == experts and sum(g) == n - 3 and min(g) >= 0
