"""What the library plans for a cache call, asked of the built library by a small host program (no GPU)."""
import os
import subprocess

import pytest

from sparse_rank_attention_block_b200 import build

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "host_checks", "cache_layout_check.cu")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    lib = build.build()
    out = str(tmp_path_factory.mktemp("layout") / "cache_layout_check")
    cmd = [build.nvcc(), *build.ARCH, "-O1", "-std=c++17", "-I" + build.CSRC, "-I" + build.INCLUDE, "-o", out, SRC,
           lib, "-Xlinker", "-rpath", "-Xlinker", os.path.dirname(lib)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def ask(B, H, H_kv, d, block, max_blocks, rows, max_new, weights=0):
        r = subprocess.run([out] + [str(x) for x in (B, H, H_kv, d, block, max_blocks, rows, max_new, weights)],
                           capture_output=True, text=True, check=True)
        return dict(zip(("workers", "whole_row_tiles", "wide_join", "join_ctas", "line_places"), map(int, r.stdout.split())))
    return ask


@pytest.mark.parametrize("B,H,H_kv,max_new,wide", [
    (1, 32, 8, 1, 1),                              # 296 CTAs for 8 units: 37 parts to a row
    (2, 32, 8, 1, 1), (3, 32, 8, 1, 0), (64, 32, 8, 1, 0),
    (1, 32, 8, 8, 1), (1, 32, 8, 12, 0),           # 16 units; 24
    (58000, 1024, 1024, 36, 0)])                   # 178 million units: 16 times as many do not fit 32 bits
def test_join_of_many_units_takes_a_warp_per_row(plan, B, H, H_kv, max_new, wide):
    y = plan(B, H, H_kv, 128, 32, 1024 if B < 1000 else 17, B * max_new, max_new)
    assert y["whole_row_tiles"] == 0 and y["join_ctas"] < 1 << 31
    assert y["wide_join"] == wide, y
