"""Columns that the adapters' second product gives to the tensor cores: every width is one that the MMA has, so the rule
of the kernel (a header function) is compiled and evaluated here, without a GPU."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include <cstdio>
#include "grouped_internal.h"
int main() {
    for (int pair = 0; pair < 2; ++pair)
        for (int own = 0; own <= 256; ++own)
            std::printf("%d %d %d\n", pair, own, cf::lora_tensor_columns(own, pair != 0));
    const int sizes[] = {17, 33, 255, 257, 1000, 100000, (1 << 30) + 7, 0x7fffffff - (1 << 23), 0x7fffffff - 511};
    for (int step = 16; step <= 32; step *= 2)
        for (int bn = step > 16 ? 128 : 16; bn <= 256; bn *= 2)
            for (int rows : sizes) {
                const int tiles = int((static_cast<long long>(rows) + bn - 1) / bn);
                if (tiles > 1)
                    std::printf("cut %d %d %d %d\n", bn, rows, tiles, cf::grouped_rows_per_tile(rows, tiles, step));
            }
    for (int kind = cf::GR_FORWARD; kind <= cf::GR_LORA; ++kind)
        std::printf("step %d %d %d\n", kind, cf::grouped_column_step(kind, false), cf::grouped_column_step(kind, true));
}
"""


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    d = tmp_path_factory.mktemp("columns")
    (d / "columns.cpp").write_text(SOURCE)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    gxx = shutil.which("g++")
    assert gxx, "no g++"
    subprocess.run([gxx, "-std=c++17", "-I", os.path.join(cuda, "include"), "-I",
                    os.path.join(ROOT, "memory_fusion_gb300", "csrc"), str(d / "columns.cpp"), "-o", str(d / "columns")],
                   check=True)
    return subprocess.run([str(d / "columns")], check=True, capture_output=True, text=True).stdout.splitlines()


def test_tensor_core_columns_are_widths_of_the_mma(lines):
    """N of one CTA's MMA (M = 128) is a multiple of 16, of a pair's (M = 256) one of 32; no row is lost to rounding up."""
    rows = [tuple(int(v) for v in ln.split()) for ln in lines if ln[0].isdigit()]
    assert len(rows) == 2 * 257
    for pair, own, nx in rows:
        step = 32 if pair else 16
        assert nx % step == 0 and own - step < nx <= own, (pair, own, nx)


def test_steps(lines):
    for ln in lines:
        if ln.startswith("step"):
            single, pair = (int(v) for v in ln.split()[2:])
            assert single % 16 == 0 and pair % 32 == 0, ln


def test_row_tiles_hold_a_groups_rows(lines):
    """Tiles of equal size up to the largest number of rows a call may have: none wider than the accumulator, none empty,
    together all rows."""
    cuts = [tuple(int(v) for v in ln.split()[1:]) for ln in lines if ln.startswith("cut")]
    assert len(cuts) >= 50
    for bn, rows, tiles, per in cuts:
        assert 0 < per <= bn and per * (tiles - 1) < rows <= per * tiles, (bn, rows, tiles, per)


def test_every_load_of_tensor_memory_has_a_wait_that_names_its_registers():
    """A wait without operands does not keep arithmetic on the loaded registers behind it: each load into a register
    array is followed by a wait that has the array as operand."""
    with open(os.path.join(ROOT, "memory_fusion_gb300", "csrc", "gemm_grouped.cu")) as f:
        text = f.read()
    loads = list(re.finditer(r"ptx::tmem_ld(?:32|_blocks)\([^;]*?, (v(?:\[\d\])?)\);", text))
    assert len(loads) >= 6
    for m in loads:
        wait = re.search(r"ptx::tmem_ld_wait\(" + re.escape(m.group(1)) + r"\);", text[m.end():m.end() + 250])
        assert wait, text[m.start():m.end() + 80]
    assert "tmem_ld_wait()" not in text
