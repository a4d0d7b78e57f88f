"""CPU checks of the embedding, the experts' products and the gated activation
with its 8-bit checkpoint: their C entry points under the host sanitizers
(tests/host_fake/model_driver.cpp: every refused call launches nothing), every
launch of their launchers (tests/host_fake/model_launch_driver.cpp), and the
refusals of the torch binding that need no GPU."""

import os
import shutil
import subprocess

import pytest
import torch

import ring_allreduce_rs_amd as ar

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "ring_allreduce_rs_amd", "csrc")
FAKE = os.path.join(ROOT, "tests", "host_fake")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/llvm/bin/clang++"
SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
       "-Xarch_host", "-fno-sanitize-recover=all"]


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)),
                    reason="needs the ROCm toolchain")
@pytest.mark.parametrize("driver,sources", [
    ("model_driver.cpp", ()),
    ("model_launch_driver.cpp", ("embed.hip", "product.hip", "gate.hip"))])
def test_under_sanitizers(tmp_path, driver, sources):
    common = ["-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-x", "hip",
              "--cuda-host-only", f"-I{ROOT}/include", f"-I{CSRC}", f"-I{FAKE}"] + SAN
    objs = []
    for src in (*(os.path.join(CSRC, f) for f in ("ar_api.cpp", "model_api.cpp", "dispatch.hip",
                                                  *sources)),
                os.path.join(FAKE, "fake_hip.cpp"), os.path.join(FAKE, driver)):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        r = subprocess.run([HIPCC] + common + ["-c", src, "-o", obj],
                           capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, f"compile {src}:\n{r.stderr[-4000:]}"
        objs.append(obj)
    exe = str(tmp_path / "driver")
    # (the device code that the host objects name is not there and not asked for)
    r = subprocess.run([CLANG, "-fsanitize=address,undefined", "-no-pie",
                        "-Wl,--unresolved-symbols=ignore-all", "-o", exe] + objs,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, f"link:\n{r.stderr[-4000:]}"
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "ALL OK" in r.stdout, (r.stdout + r.stderr)[-6000:]


X = torch.randn(6, 64)
IDS = torch.zeros(6, dtype=torch.int64)
W = torch.randn(3, 64, 64)
AT = torch.arange(6, dtype=torch.int32)
PLAN = ar.ExpertPlan(AT.view(-1, 1), AT, torch.tensor([0, 2, 2, 6], dtype=torch.int32))
SAVED = ar.Saved8(torch.zeros((6, 2, 64), dtype=torch.int8), torch.ones((6, 2, 2), dtype=torch.uint8))
# every operator, by the tensor that it looks at first
CALLS = {
    "embedding": (lambda t: ar.embedding(t, IDS), X),
    "embedding_backward": (lambda d: ar.embedding_backward(d, IDS, 9), X),
    "expert_matmul": (lambda r: ar.expert_matmul(r, W, PLAN), X),
    "expert_matmul_drows": (lambda d: ar.expert_matmul_drows(d, W, PLAN), X),
    "expert_matmul_dweights": (lambda d: ar.expert_matmul_dweights(d, X, PLAN), X),
    "save_8bit": (lambda x: ar.save_8bit(x), X),
    "silu_gate": (lambda h: ar.silu_gate(h), X),
    "silu_gate_backward": (lambda d: ar.silu_gate_backward(d, SAVED), X),
}


@pytest.mark.parametrize("name", CALLS)
def test_gradients_are_not_lost(name):
    call, arg = CALLS[name]
    leaf = arg.clone().requires_grad_()
    for t in (leaf, leaf * 2):
        with pytest.raises(ValueError, match="requires grad"):
            call(t)
        with torch.no_grad(), pytest.raises(ValueError, match="not on a GPU"):
            call(t)
    with pytest.raises(ValueError, match="not on a GPU"):
        call(arg)
    with pytest.raises(ValueError, match="unsupported dtype"):
        call(arg.half())
    with pytest.raises(ValueError, match="not a tensor"):
        call([1.0])


def test_checkpoints_off_the_gpu():
    with pytest.raises(ValueError, match="not on a GPU"):
        ar.restore_8bit(SAVED)
    assert ar.AR_SAVE_GROUP == 32


def test_names():
    names = {"embedding", "embedding_backward", "expert_matmul", "expert_matmul_drows",
             "expert_matmul_dweights", "Saved8", "save_8bit", "restore_8bit", "silu_gate",
             "silu_gate_backward"}
    assert names <= set(dir(ar)) and all(callable(getattr(ar, n)) for n in names)
