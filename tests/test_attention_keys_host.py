"""CPU checks of csrc/attention_keys.h, the integer arithmetic with which the
paged attention finds a row's keys and a wave's first tile of them, compiled
as plain C++ (signed overflow wraps, as it does on the GPU): lengths up to
2^31 - 1, in rows of the block table that are much shorter."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_token_amd", "csrc")
TOP = 2 ** 31 - 1

SOURCE = r"""
#include "attention_keys.h"
using namespace gdn;
extern "C" void range_of(int causal, int window, int n, int len, int L, int i, int *out) {
    key_range(causal, window, Request{0, n, len, L}, i, out[0], out[1]);
}
// the keys that the rows of tokens i0 .. i1 see, their splits, and of split
// `split` its keys and where wave `wave` begins
extern "C" void share_of(int causal, int window, int n, int len, int L, int i0, int i1, int chunk, int splits, int split,
                         int tile, int wave, int *out) {
    const Request r{0, n, len, L};
    int lo, hi, x;
    key_range(causal, window, r, i0, lo, x);
    key_range(causal, window, r, i1, x, hi);
    const Splits s = splits_of(lo, hi, chunk, splits);
    const int k_lo = lo > split * chunk ? lo : split * chunk;
    out[0] = s.first;
    out[1] = s.last;
    out[2] = k_lo;
    out[3] = split == splits - 1 || hi < (split + 1) * chunk ? hi : (split + 1) * chunk;
    out[4] = first_tile(k_lo, tile, wave);
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("attention_keys")
    (d / "keys.cpp").write_text(SOURCE)
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-fwrapv", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(d / "keys.cpp"),
                           "-o", str(d / "keys.so")])
    return ctypes.CDLL(str(d / "keys.so"))


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("L", [0, 1, 37, 64])
def test_a_rows_keys(lib, causal, L):
    """The keys that the mask leaves, wherever the request ends."""
    out = (ctypes.c_int * 2)()
    for length in [L, L + 1, L + 63, 2 ** 20, TOP - 64, TOP] if L == 64 else [L]:
        for n in (1, 2, 40):
            for window in (0, 1, 2, 63, 64, 1000, TOP):
                for i in {0, n // 2, n - 1}:
                    p = length - n + i
                    lib.range_of(causal, window, n, length, L, i, out)
                    seen = [j for j in range(L) if (not causal or j <= p) and (not window or j > p - window)]
                    assert list(range(out[0], out[1])) == seen
                    assert 0 <= out[0] <= max(L, 0) and out[1] <= L


@pytest.mark.parametrize("tile,waves", [(64, 8), (32, 8), (64, 4), (64, 1)])
@pytest.mark.parametrize("length", [TOP, TOP - 63, TOP - 447, TOP - 512, 2 ** 30, 100])
def test_tiles_begin_at_keys_that_exist(lib, tile, waves, length):
    """A request that is longer than its row: no wave's first tile lies below key 0, and one
    at or past the last key is not taken."""
    out = (ctypes.c_int * 5)()
    for L in (16, 80, 4096, TOP - 1024):
        L = min(L, length)
        for causal in (0, 1):
            for window in (0, 1, 7, 100, 447, 448, 5000):
                for n in (1, 3):
                    for chunk, splits in ((0x40000000, 1), (1024, 3), (8388608, 256)):
                        for split in (0, splits - 1):
                            for wave in range(waves):
                                lib.share_of(causal, window, n, length, L, 0, n - 1, chunk, splits, split, tile, wave, out)
                                first, last, k_lo, k_hi, j0 = out
                                if split != first and not first <= split <= last:
                                    continue
                                assert 0 <= j0 <= TOP - 512 and k_lo <= max(L, split * chunk) and k_hi <= L
