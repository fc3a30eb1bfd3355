"""Indexes that the kernels load by, compiled for the host and driven over every
length: no load lies outside its buffer."""
import os
import subprocess

from point_cloud_tokenization_amd import build as fbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _run(tmp_path, name):
    exe = str(tmp_path / name)
    subprocess.run([fbuild.hipcc(), "--cuda-host-only", "-x", "hip", "-std=c++17", "-O1",
                    "-Wno-everything", "-I", os.path.join(ROOT, "include"), "-I", fbuild.CSRC,
                    "-o", exe, os.path.join(ROOT, "tests", name + ".hip")],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout[-200:] + r.stderr
    return r.stdout


def test_walk_over_the_plane(tmp_path):
    """Sequences that end in the first half of a tile of 64 keys, in the plane's last
    row: the second block of a pair is not loaded from behind the plane."""
    assert "walks ok" in _run(tmp_path, "plane_walk_main")


def test_parts_of_the_gates(tmp_path):
    """The parts of a gate's gradient, for boundaries in order (each part of a
    sequence, once) and for ones that run backwards (none outside the parts)."""
    assert "parts ok" in _run(tmp_path, "gate_parts_main")
