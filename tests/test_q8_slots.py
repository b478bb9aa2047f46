"""Slots of page-table entries on the CPU (the library's header compiled with
the host compiler): every entry gives a slot in its page, or one that no append
takes for padding or for a place in a pool."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_attention_long_anchor_b200", "csrc")


def test_slots_of_entries_that_no_pool_has(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    cases = []
    for ps in (4, 6, 12):
        top = (2 ** 31 - 1) >> ps
        cases += [(e, r, ps) for e in (0, 1, 17, top - 1, top, top + 1, 2 * top + 1, 2 ** 26 + 3, 2 ** 28 + 1, 2 ** 31 - 1, -1, -2, -7, -2 ** 31)
                  for r in (0, 1, (1 << ps) - 1)]
    src = tmp_path / "t.cpp"
    src.write_text('#include <cstdio>\n#include "q8_index.h"\nint main() {\n  static const long long c[][3] = {%s};\n'
                   '  for (auto& x : c) {\n    const int s = kascade::q8_slot((int)x[0], (unsigned)x[1], (int)x[2]);\n'
                   '    std::printf("%%d %%d\\n", s, (int)kascade::q8_slot_ok(s, (int)(0x7fffffffu >> x[2]), (int)x[2]));\n  }\n}\n'
                   % ", ".join("{%d,%d,%d}" % c for c in cases))
    exe = tmp_path / "t"
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = list(map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()))
    for (e, r, ps), slot, inside in zip(cases, out[::2], out[1::2]):
        if 0 <= e <= (2 ** 31 - 1) >> ps:
            assert slot == (e << ps) + r and slot >= 0
            assert inside == (e < (2 ** 31 - 1) >> ps)      # the largest pool has one page less
        else:
            assert slot == -2 ** 31 and not inside
