"""The turns of a ring of stages that a kernel waits for when it gives up or ends."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_open_turns_are_the_ones_in_flight(tmp_path):
    exe = tmp_path / "turns"
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror",
                    "-I", os.path.join(ROOT, "ring_allreduce_reducescatter_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "csrc", "turns.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
