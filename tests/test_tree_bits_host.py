"""The masks of a tree's attention on the CPU: the kernel's own function (csrc/tree_bits.h), asked for every row of a
tile as the kernel does, reads the words of nodes in use only and gives the bits that the sets name."""
import os
import subprocess

from self_speculative_sparse_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_rows_read_the_words_of_their_sequences_nodes_only(tmp_path):
    exe = str(tmp_path / "tree_bits_check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", build.CSRC, os.path.join(HERE, "tree_bits_check.cpp"), "-o", exe],
                   check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
