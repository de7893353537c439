"""Compiles a host program against the kernels' CUDA-free headers."""
import os
import shutil
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mixture_experts_layer_18_gb300", "csrc")


def compile_host(tmp_path, source):
    """Path of the program compiled from `source`."""
    cxx = shutil.which("g++")
    assert cxx, "the library's build needs g++ too"
    src, exe = tmp_path / "check.cpp", tmp_path / "check"
    src.write_text(source)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    return str(exe)
