"""The paged logits' pipeline as a model on the host: what is under way when a CTA gives up."""
import os
import subprocess

from fp8_mqa_logits_02_gb300 import nvcc_build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_no_copy_lands_after_the_end(tmp_path):
    exe = str(tmp_path / "model")
    cmd = [nvcc_build.nvcc_path(), "-O2", "-std=c++17", *nvcc_build.ARCH_FLAGS, "-I", nvcc_build.CSRC, "-o", exe,
           os.path.join(HERE, "paged_logits_model.cu")]
    built = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert built.returncode == 0, built.stdout
    ran = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=300)
    assert ran.returncode == 0, ran.stdout
