"""CPU checks of what the grouped products do on the host."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

INVALID = 1


def test_the_unread_workspace_is_the_librarys(moelib, monkeypatch):
    """A call without a workspace writes to memory that no allocator hands out: a
    block of the caching allocator may have an earlier owner whose work on the
    stream it was freed on is still to come, and these calls run on any stream."""
    import moe_expert_layer_08_b200 as m
    asked = []

    class Library:
        @staticmethod
        def moe_grouped_unread_workspace(device, where):
            asked.append(device)
            where._obj.value = 0x70000 + 0x1000 * device
            return 0

    def no_allocator(*args, **kwargs):
        raise AssertionError("memory of the allocator")

    monkeypatch.setattr(m, "_unread", {})
    monkeypatch.setattr(m, "load", lambda: Library)
    for name in ("empty", "zeros", "full"):
        monkeypatch.setattr(torch, name, no_allocator)
    for device in (0, 1, 0):
        at, size = m._grouped_workspace(None, torch.device("cuda", device))
        assert at == 0x70000 + 0x1000 * device and size == m._GROUPED_WORKSPACE
    assert asked == [0, 1]


def test_unread_workspace_refusals(moelib):
    p = ctypes.c_void_p()
    assert moelib.moe_grouped_unread_workspace(-1, ctypes.byref(p)) == INVALID
    assert moelib.moe_grouped_unread_workspace(0, None) == INVALID
    assert p.value is None


CHUNKS = r"""
#include <cstdio>
#include "row_chunks.h"

int main() {
    const int top = 2147483647 - 65535;  // rows of a call, at most
    const int widths[] = {64, 160, 256};
    for (int most : widths) {
        const int ends[] = {1, most, 1000 * most, top};
        for (int end : ends)
            for (int i = -70000; i <= 70000; ++i) {
                const long long want = (long long)end + i;
                if (want < 1 || want > top) continue;
                const int rows = int(want);
                const moe::RowChunks c = moe::row_chunks(rows, most);
                const long long count = c.count, size = c.size;
                if (count != (want + most - 1) / most || size % 16 || size < 16 || size > most ||
                    (count - 1) * size >= want || count * size < want || (size - 16) * count >= want) {
                    std::printf("%d rows of %d: %d of %d\n", rows, most, c.count, c.size);
                    return 1;
                }
            }
    }
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_row_chunks_at_every_size(tmp_path):
    """Rows are cut into as few chunks as hold them, none empty, up to the largest
    number of rows that a call accepts (undefined overflows end the program)."""
    src, exe = tmp_path / "chunks.cpp", tmp_path / "chunks"
    src.write_text(CHUNKS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-Wall", "-Werror",
                    "-I", os.path.join(ROOT, "moe_expert_layer_08_b200", "csrc"), str(src), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    done = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert done.returncode == 0, done.stdout + done.stderr
