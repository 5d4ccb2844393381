"""The window's arithmetic that the kernels share, without a GPU: compiled here as plain C++
with checks for overflow, against the mask's definition."""
import ctypes
import os
import subprocess

import pytest

from tests import _plain

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MOST = 2 ** 31 - 1

SHIM = r'''
#include "fa_window.h"
using namespace fa;
extern "C" {
int t_hides(int n, int w, int s) { return window_hides(n, w, s); }
int t_window(int n, int w, int s) { return cut_window(n, w, s).window; }
int t_sinks(int n, int w, int s) { return cut_window(n, w, s).sinks; }
int t_blocks(int s, int win, int block) { return sink_blocks(s, win, block); }
uint32_t t_span(int lo, int hi) { return span(lo, hi); }
}
'''


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    d = tmp_path_factory.mktemp("window")
    src, lib = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", "-static-libubsan",
                    "-I", os.path.join(ROOT, "exact_io_aware_12_gb300", "csrc"), str(src), "-o", str(lib)], check=True)
    L = ctypes.CDLL(str(lib))
    L.t_span.restype = ctypes.c_uint32
    return L


SIZES = (1, 2, 7, 29, 30, 31, 60, MOST - 126, MOST)


@pytest.mark.parametrize("N", [1, 2, 30])
def test_cut_windows_show_the_same_keys(shim, N):
    for w in SIZES:
        for s in (0,) + SIZES:
            # (the definition on numbers of any size)
            want = [[j <= i and (j > i - w or j < s) for j in range(N)] for i in range(N)]
            assert _plain.visible(N, N, shim.t_window(N, w, s), shim.t_sinks(N, w, s)).tolist() == want
            assert bool(shim.t_hides(N, w, s)) == any(not want[i][j] for i in range(N) for j in range(i + 1))
        assert shim.t_hides(N, 0, w) == 0 and shim.t_window(N, 0, w) == 0


def test_sink_blocks_hold_the_sinks_before_the_window(shim):
    """After the cut, of any length that the kernels take (65535 blocks of 128)."""
    for N in (1, 128, 129, 1000, 65535 * 128):
        for w in SIZES:
            for s in SIZES:
                sinks = shim.t_sinks(N, w, s)
                for win in (0, 1, 3, (N - 1) // 128):
                    n = shim.t_blocks(sinks, win, 128)
                    assert n == min(-(-sinks // 128), win) and 0 <= n <= win


def test_spans_up_to_their_widest(shim):
    """Also the whole range of a sink's queries, 2^31 wide: no signed overflow."""
    ends = (-2 ** 30, -2 ** 30 + 1, -200, -1, 0, 1, 127, 2 ** 30 - 1, 2 ** 30)
    for lo in ends:
        for hi in ends:
            n = shim.t_span(lo, hi)
            assert n == max(0, hi - lo)
            for x in (0, 1, 64, 127):   # (the kernel's compare of columns of a tile)
                assert ((x - lo) % 2 ** 32 < n) == (lo <= x < hi)
