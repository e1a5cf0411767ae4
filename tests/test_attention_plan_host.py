"""CPU checks of csrc/attention_plan.h, compiled as plain C++: a call's plan never
needs more workspace than its workspace size function says, which does not know
the window, and its parts cover the keys that max_seq_len allows."""
import ctypes
import itertools
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_token_amd", "csrc")
SOURCE = r"""
#include "attention_plan.h"
using namespace gdn;
extern "C" void plan(int min_chunk, int idle_chunk, int many_chunk, int waves, int room, int many_rows, long long T, long long S,
                     int hq, int hk, int d, int longest, int window, long long *out) {
    const Plan p = plan_of({min_chunk, idle_chunk, many_chunk, waves, room, many_rows}, T, S, hq, hk, d, longest, window);
    const Launch *l[2] = {&p.few, &p.many};
    for (int i = 0; i < 2; ++i) {
        out[5 * i] = l[i]->units;
        out[5 * i + 1] = l[i]->rows;
        out[5 * i + 2] = l[i]->chunk;
        out[5 * i + 3] = l[i]->splits;
        out[5 * i + 4] = l[i]->floats;
    }
}
"""
RULES = {"kv8": (1024, 512, 256, 8, 512, 128), "kv4": (1024, 512, 256, 4, 512, 128), "kv4 of 256": (1024, 512, 256, 4, 512, 64)}


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("attention_plan")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(d / "plan.cpp"),
                           "-o", str(d / "plan.so")])
    lib = ctypes.CDLL(str(d / "plan.so"))
    i32, i64 = ctypes.c_int32, ctypes.c_int64
    lib.plan.argtypes = [i32] * 6 + [i64, i64] + [i32] * 5 + [ctypes.POINTER(i64)]
    return lib


def plan(lib, rules, *sizes):
    out = (ctypes.c_int64 * 10)()
    lib.plan(*RULES[rules], *sizes, out)
    names = ("units", "rows", "chunk", "splits", "floats")
    return [dict(zip(names, out[5 * i:5 * i + 5])) for i in range(2)]


CALLS = [(1, 1), (2, 2), (2, 5), (5, 5), (32, 32), (200, 200), (3, 1), (70, 3), (2048, 32), (8192, 1), (100, 99)]
HEADS = [(1, 1), (16, 4), (32, 8), (20, 1), (8, 8)]
LONGEST = [1, 100, 511, 512, 1000, 1023, 1024, 1025, 2047, 2048, 5000, 131072, 2 ** 31 - 1]


@pytest.mark.parametrize("rules", list(RULES))
def test_a_window_needs_no_more_workspace(lib, rules):
    for (T, S), (hq, hk), longest in itertools.product(CALLS, HEADS, LONGEST):
        size = sum(p["floats"] for p in plan(lib, rules, T, S, hq, hk, 128, longest, 0))
        for window in (1, 100, 511, 512, 513, 1023, 1024, 1025, 2048, 10000, 2 ** 31 - 1):
            few, many = plan(lib, rules, T, S, hq, hk, 128, longest, window)
            assert few["floats"] + many["floats"] <= size, (T, S, hq, hk, longest, window)
            if window <= RULES[rules][0]:
                assert few["splits"] <= 1, (T, S, hq, hk, longest, window)


@pytest.mark.parametrize("rules", list(RULES))
def test_parts_cover_the_keys(lib, rules):
    for (T, S), (hq, hk), longest in itertools.product(CALLS, HEADS, LONGEST):
        for p in plan(lib, rules, T, S, hq, hk, 128, longest, 0):
            assert p["splits"] <= 1 or (p["splits"] - 1) * p["chunk"] < longest <= p["splits"] * p["chunk"]
            assert p["floats"] == (p["rows"] * p["splits"] * 130 if p["splits"] > 1 else 0)
