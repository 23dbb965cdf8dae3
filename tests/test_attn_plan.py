"""The workspace of decode attention against what a call takes: both from the
host's planning header, compiled here with g++."""
import ctypes
import os
import subprocess

import pytest

from rank_gemm_amd import lora

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rank_gemm_amd", "csrc")

SOURCE = """
#include "attn_plan.h"
extern "C" {
size_t used(int B, int heads, int kv, int dim, int width, int page_rows, int window, int f8, int adjacent, int* wgs) {
    const lora::AttnLayout l = lora::attn_layout(B, heads, kv, dim, width, page_rows, window, f8, adjacent);
    *wgs = l.s.wgs;
    return l.bytes;
}
size_t asked(int B, int heads, int kv, int dim, int width, int page_rows) {
    return lora::attn_workspace_bytes(B, heads, kv, dim, width, page_rows);
}
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, so = d / "plan.cpp", d / "plan.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(src), "-o",
                    str(so)], check=True)
    L = ctypes.CDLL(str(so))
    L.used.argtypes = [ctypes.c_int] * 9 + [ctypes.POINTER(ctypes.c_int)]
    L.asked.argtypes = [ctypes.c_int] * 6
    L.used.restype = L.asked.restype = ctypes.c_size_t
    return L


HEADS = [(32, 8, 128), (16, 4, 256), (64, 2, 128), (32, 8, 64), (8, 4, 32), (4, 4, 16), (70, 1, 256), (128, 2, 64),
         (12, 2, 80), (17, 17, 128), (130, 2, 128)]


@pytest.mark.parametrize("heads,kv,dim", HEADS)
def test_no_window_takes_more_than_was_asked(plan, heads, kv, dim):
    """Tables at and beside the path limits (512, 1536 and 2048 positions), windows
    from the first tile's border below them to past the table's size."""
    wgs, split = ctypes.c_int(), set()
    for B in (1, 2, 3, 15, 16, 17, 31, 32, 64, 128, 700):
        for page in (1, 16, 24):
            for limit in (512, 1536, 2048):
                for width in range(max(1, (limit - 20) // page), (limit + 40) // page + 1):
                    most = width * page
                    asked = plan.asked(B, heads, kv, dim, width, page)
                    for window in (0, 1, 100, *range(max(1, most - 34), most + 3), 2 ** 31 - 1):
                        for f8 in (0, 1):
                            for adjacent in (0, 1):
                                used = plan.used(B, heads, kv, dim, width, page, window, f8, adjacent,
                                                 ctypes.byref(wgs))
                                assert used <= asked, (B, most, window, f8, adjacent, wgs.value)
                                assert (used > 0) == (wgs.value > 0)
                                split.add(wgs.value > 0)
    assert split == {False, True}


def test_the_library_asks_for_it(plan):
    """lora_attn_decode_workspace_bytes is the same function; bytes that a split
    call needs are there and a whole row's are not."""
    L = lora.lib()
    seen = set()
    for heads, kv, dim in HEADS:
        for B in (1, 16, 300):
            for width, page in ((1, 16), (96, 16), (97, 16), (128, 16), (129, 16), (32, 16), (33, 16), (85, 24), (86, 24),
                                (4096, 64)):
                n = L.lora_attn_decode_workspace_bytes(B, heads, kv, dim, width, page)
                assert n == plan.asked(B, heads, kv, dim, width, page)
                seen.add(n > 0)
    assert seen == {False, True}
    assert L.lora_attn_decode_workspace_bytes(2, 4, 2, 64, 1 << 16, 16) > 0
    assert L.lora_attn_decode_workspace_bytes(1, 32, 8, 128, 96, 16) == 0
