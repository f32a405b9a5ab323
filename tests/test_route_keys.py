"""What the router decides from float32 keys, compiled for the host: no GPU needed."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = """
#include "route_keys.hpp"
extern "C" {
int c_none() { return tsm::kNone; }
int c_ordered(float f) { return tsm::ordered(f); }
int c_near_limit(int least, float error) { return tsm::near_limit(least, error); }
int c_group_of(int e, int size) { return (int)tsm::group_of(e, tsm::group_magic(size)); }
}
"""


@pytest.fixture(scope="module")
def keys(tmp_path_factory):
    d = tmp_path_factory.mktemp("route_keys")
    (d / "k.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "tiled_shared_memory_amd", "csrc"), str(d / "k.cpp"), "-o", str(d / "k.so")],
                   check=True)
    lib = ctypes.CDLL(str(d / "k.so"))
    lib.c_ordered.argtypes = [ctypes.c_float]
    lib.c_near_limit.argtypes = [ctypes.c_int, ctypes.c_float]
    return lib


def test_near_keys_are_keys_of_experts(keys):
    """What may be as near as the smallest chosen key reaches that key, and never -inf, the key of places that hold no
    expert (whose logits would lie past a row): float32's lowest value as a bias and infinite ones among the keys."""
    top = float(np.finfo(np.float32).max)
    for key in (-top, -3.4e38, float(np.finfo(np.float16).min), -1.0, 0.0, 0.5, 7.0, top, np.inf):
        least = keys.c_ordered(key)
        for error in (2.0 ** -27, 2.0 ** -21, 1.0, np.inf, np.nan):
            near = keys.c_near_limit(least, error)
            assert keys.c_none() < near <= least, (key, error)
    assert keys.c_near_limit(keys.c_ordered(1.0), 0.0) == keys.c_ordered(1 - 2.0 ** -22)


def test_the_group_of_every_expert(keys):
    """Of every layout of up to 512 experts."""
    wrong = [(size, e) for size in range(1, 513) for e in range(512) if keys.c_group_of(e, size) != e // size]
    assert not wrong, f"{len(wrong)}: {wrong[:8]}"
