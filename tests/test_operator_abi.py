"""CPU checks of the training operators: their C entry points under the host
sanitizers (tests/host_fake/ops_driver.cpp: every refused call launches
nothing, every accepted one launches what its arguments say), and the
refusals of the torch binding that need no GPU."""

import os
import shutil
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "ring_allreduce_rs_amd", "csrc")
FAKE = os.path.join(ROOT, "tests", "host_fake")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/llvm/bin/clang++"
SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
       "-Xarch_host", "-fno-sanitize-recover=all"]


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)),
                    reason="needs the ROCm toolchain")
def test_entry_points_under_sanitizers(tmp_path):
    common = ["-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-x", "hip",
              "--cuda-host-only", f"-I{ROOT}/include", f"-I{CSRC}", f"-I{FAKE}"] + SAN
    objs = []
    for src in (os.path.join(CSRC, "ar_api.cpp"), os.path.join(CSRC, "ops_api.cpp"),
                os.path.join(CSRC, "dispatch.hip"), os.path.join(FAKE, "fake_hip.cpp"),
                os.path.join(FAKE, "ops_driver.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        r = subprocess.run([HIPCC] + common + ["-c", src, "-o", obj],
                           capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, f"compile {src}:\n{r.stderr[-4000:]}"
        objs.append(obj)
    exe = str(tmp_path / "ops_driver")
    r = subprocess.run([CLANG, "-fsanitize=address,undefined", "-o", exe] + objs,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, f"link:\n{r.stderr[-4000:]}"
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and "ALL OK" in r.stdout, (r.stdout + r.stderr)[-6000:]


def test_tensors_off_the_gpu_are_refused():
    import ring_allreduce_rs_amd as ar
    x = torch.randn(4, 32)
    stat, ids = torch.zeros(4), torch.zeros((4, 2), dtype=torch.int64)
    plan = ar.ExpertPlan(ids.int(), ids.int().view(-1), torch.zeros(4, dtype=torch.int32))
    for call in (lambda: ar.layer_norm(x), lambda: ar.layer_norm_backward(x, x, stat, stat),
                 lambda: ar.expert_dispatch(x, ids, 3),
                 lambda: ar.expert_combine(x.repeat(2, 1), torch.zeros(4, 2), plan),
                 lambda: ar.expert_dispatch_backward(x.repeat(2, 1), plan),
                 lambda: ar.expert_combine_backward(x, x.repeat(2, 1), torch.zeros(4, 2), plan),
                 lambda: ar.distill_loss(x, ids, torch.zeros(4, 2)),
                 lambda: ar.distill_backward(stat, x, ids, torch.zeros(4, 2), stat),
                 lambda: ar.distill_step(stat, x, ids, torch.zeros(4, 2))):
        with pytest.raises(ValueError, match="not on a GPU"):
            call()


def test_the_binding_says_what_to_build(tmp_path):
    # a copy without _torch_ops.so must raise when an operator is asked for
    pkg = tmp_path / "ring_allreduce_rs_amd"
    shutil.copytree(os.path.join(ROOT, "ring_allreduce_rs_amd"), pkg,
                    ignore=shutil.ignore_patterns("_torch_ops*", "__pycache__", "csrc"))
    code = ("import sys; sys.path.insert(0, %r)\n"
            "import ring_allreduce_rs_amd as ar\n"
            "try:\n ar.layer_norm\nexcept ImportError as e:\n print('RAISED', e)\n"
            % str(tmp_path))
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert "RAISED" in out.stdout and "_build.py" in out.stdout, out.stdout + out.stderr
