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
int c_near_groups(float error, float a1, float a2, float b1, float b2) {
  return tsm::near_sums(b1 + b2, a1 + a2, tsm::group_tolerance(error, a1, a2)) ||
         tsm::near_sums(a1 + a2, b1 + b2, tsm::group_tolerance(error, b1, b2));
}
float c_group_sum(float b1, float b2) { return tsm::group_sum(b1, b2); }
float c_group_tolerance(float error, float b1, float b2) { return tsm::group_tolerance(error, b1, b2); }
int c_near_sums(float o, float b1, float b2, float error) {
  return tsm::near_sums(o, tsm::group_sum(b1, b2), tsm::group_tolerance(error, b1, b2));
}
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
    lib.c_near_groups.argtypes = [ctypes.c_float] * 5
    lib.c_group_sum.argtypes, lib.c_group_sum.restype = [ctypes.c_float] * 2, ctypes.c_float
    lib.c_group_tolerance.argtypes, lib.c_group_tolerance.restype = [ctypes.c_float] * 3, ctypes.c_float
    lib.c_near_sums.argtypes = [ctypes.c_float] * 4
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


@pytest.mark.parametrize("size", [0.0, 0.1, 16.0, 1000.0, 1e6, 1e30])
@pytest.mark.parametrize("error", [2.0 ** -27, 2.0 ** -21])
def test_groups_in_the_other_order_are_near(keys, size, error):
    """Two groups' sums of two keys, biases of either sign that all but cancel: where the exact sums are not in the order of
    the float32 ones, one of the two groups finds the other near."""
    rng = np.random.default_rng(int(size) + 3)
    other = 0
    for _ in range(4000):
        s = rng.random((2, 2)) * 2.0 ** -8  # exact scores, and float32 ones off by less than `error`
        s32 = (s + (rng.random((2, 2)) - 0.5) * 1.9 * error).astype(np.float32)
        b = np.zeros((2, 2), np.float32)
        b[:, 0] = size * (1 + rng.random(2))
        b[:, 1] = -(b[:, 0].astype(np.float64) + s.sum(1))  # (the sums are what this rounding leaves, and a little)
        b[1, 1] = np.float32(b[1, 1] + (rng.random() - 0.5) * 2.0 ** -23)
        k32 = s32 + b
        exact, got = (s + b.astype(np.float64)).sum(1), k32[:, 0] + k32[:, 1]
        assert k32.dtype == got.dtype == np.float32
        if np.sign(exact[1] - exact[0]) != np.sign(got[1] - got[0]):
            other += 1
            assert keys.c_near_groups(error, *map(float, k32.ravel())), (s, b)
    # (without biases the exact sums are too far apart for it; at 1e30 float64 too holds nothing of the scores)
    assert other > 20 or size in (0.0, 1e30)


def test_sums_past_the_range_of_float32(keys):
    """A group of experts is one also where its sum passes float32's range (a mask of its lowest value twice); what then
    reads as equal is near, at a finite distance, and a group of none stays one."""
    top, f = float(np.finfo(np.float32).max), keys.c_group_sum
    assert f(-np.inf, 0.0) == -np.inf and f(0.5, 0.25) == 0.75 and f(-top, 0.0) == -top
    assert f(np.inf, 0.0) == f(np.inf, 1.0) == f(np.inf, np.inf) == f(np.inf, -top) == np.inf > f(top, top)
    pairs = [(-top, -top), (-top, 0.0), (0.25, -top), (-3e38, -1e38), (-3e38, -0.9e38), (-2e38, -1e38), (0.5, 0.25),
             (top, 0.0), (top, top), (3e38, 2e38), (top, -top)]
    for a in pairs:
        assert np.isfinite(f(*a)), a
        assert np.isfinite(keys.c_group_tolerance(2.0 ** -21, *a)), a
        for b in pairs:
            exact, got = sum(a) - sum(b), np.float64(f(*a)) - np.float64(f(*b))
            assert np.sign(exact) == np.sign(got) or abs(got) <= keys.c_group_tolerance(2.0 ** -21, *a), (a, b)


def test_a_group_of_none_is_near_nothing(keys):
    """Groups without an expert to choose (out of service, or only there to fill up a power of two) decide nothing; nor
    does one of an infinite bias, unless the other has one too."""
    near, top = keys.c_near_sums, float(np.finfo(np.float32).max)
    for error in (2.0 ** -27, 2.0 ** -21, 2.0 ** -9):
        for b1, b2 in ((0.5, 0.25), (1.0, 0.0), (-1e9, 0.0), (1e30, 1.0), (-top, -top), (top, top), (np.inf, 0.0),
                       (-np.inf, 0.0)):
            assert not near(-np.inf, b1, b2, error), (b1, b2)
            assert not near(keys.c_group_sum(b1, b2), -np.inf, 0.0, error), (b1, b2)
        assert not near(0.5, np.inf, 0.0, error) and not near(keys.c_group_sum(np.inf, 0.0), 0.5, 0.0, error)
        assert near(0.5, 0.25, 0.25, error)
