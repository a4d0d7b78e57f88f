"""The package's names: the collectives' come without torch and without the
operators' binding, the operators' when they are asked for."""

import os
import shutil
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code, path):
    out = subprocess.run([sys.executable, "-c", f"import sys; sys.path.insert(0, {str(path)!r})\n"
                          + code], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "OK", out.stdout + out.stderr


def test_collectives_without_torch(tmp_path):
    # torch cannot be imported, and the binding is not there
    pkg = tmp_path / "ring_allreduce_rs_amd"
    shutil.copytree(os.path.join(ROOT, "ring_allreduce_rs_amd"), pkg,
                    ignore=shutil.ignore_patterns("_torch_ops*", "__pycache__", "csrc"))
    run("sys.modules['torch'] = None\n"
        "from ring_allreduce_rs_amd import *\n"
        "assert callable(allreduce) and callable(bind) and predict_us and chunk_range\n"
        "print('OK')", tmp_path)


def test_operators_on_demand():
    run("import ring_allreduce_rs_amd as ar\n"
        "loaded = lambda: 'ring_allreduce_rs_amd.operators' in sys.modules\n"
        "assert not loaded()\n"
        "names = ['ExpertPlan', 'layer_norm', 'layer_norm_backward', 'expert_dispatch',\n"
        "         'expert_dispatch_backward', 'expert_combine', 'expert_combine_backward',\n"
        "         'distill_loss', 'distill_backward', 'distill_step']\n"
        "assert set(names) <= set(dir(ar)) and not loaded()\n"
        "assert all(callable(getattr(ar, n)) for n in names)\n"
        "from ring_allreduce_rs_amd import distill_step\n"
        "assert distill_step is ar.distill_step\n"
        "assert not hasattr(ar, 'no_such_operator')\n"
        "from ring_allreduce_rs_amd import *\n"
        "assert layer_norm is ar.layer_norm and allreduce is ar.allreduce\n"
        "print('OK')", ROOT)
