"""CPU test of the layout that the tensor-core kernel of linear attention keeps in shared memory: what it
reads 16 bytes at a time starts on 16 bytes, wherever the members before it end."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "persistent_rnn_recurrence_gb300", "csrc")


def test_tables_of_decays_start_on_16_bytes(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "layout.cpp", tmp_path / "layout"
    src.write_text("""
#include <cstdio>
#include "linear_attention_tables.h"
using prnn::Tables;
int main() {
  printf("%zu %zu %zu %zu %zu\\n", offsetof(Tables, dec), offsetof(Tables, diag), sizeof(Tables::diag[0]),
         alignof(Tables), sizeof(Tables));
}
""")
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    dec, diag, row, align, size = map(int, out.split())
    # two halves of a diagonal block's row are read at column 0 and column 16
    assert dec % 16 == 0 and diag % 16 == 0 and row % 16 == 0 and align % 16 == 0 and size % 16 == 0
