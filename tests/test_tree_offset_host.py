"""The running offset of the attention kernel's softmax (tree_offset.h), on the
host: for every magnitude of scores a row's keys end in a bounded number of
passes, with weights that binary16 holds and that keep the largest scores
apart from the rest."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "residual_add_rmsnorm_gb300", "csrc")

SOURCE = r'''
#include "tree_offset.h"
using namespace rarn::tree;
// Runs of `per` scores, as the kernel takes 32 keys: a weight is 2^(score +
// sub).  w[j]: what key j's weight has become, in log2, when all are through;
// the passes over the run that took most.
extern "C" int walk(const float *score, int n, int per, float lift, float *w) {
    const float most = kHighest - lift, centre = kCentre - lift;
    float top = -INFINITY;
    for (int j = 0; j < n && j < 2 * per; ++j) top = fmaxf(top, score[j]);
    float sub = -first_offset(top, centre);
    int worst = 0;
    for (int j0 = 0; j0 < n; j0 += per) {
        const int end = j0 + per < n ? j0 + per : n;
        int moves = 0;
        for (int passes = 1;; ++passes) {
            if (passes > worst) worst = passes;
            if (passes > 100) return passes;
            float high = -INFINITY;
            for (int j = j0; j < end; ++j) {
                w[j] = score[j] + sub;
                high = fmaxf(high, w[j]);
            }
            if (high > most && moves < kMoves) {
                ++moves;
                float down = 0.f;
                sub = moved_offset(sub, high, centre, &down);
                if (!(down == rintf(down))) return -1;
                for (int j = 0; j < j0; ++j) w[j] -= down;
                continue;
            }
            for (int j = j0; j < end; ++j) w[j] = w[j] > most ? most : w[j];
            break;
        }
    }
    return worst;
}
'''


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("offset")
    (d / "offset.cpp").write_text(SOURCE)
    lib = str(d / "offset.so")
    # no contraction: the kernel's sums are separate operations
    subprocess.run([cxx, "-O2", "-ffp-contract=off", "-shared", "-fPIC", "-I", CSRC,
                    str(d / "offset.cpp"), "-o", lib], check=True)
    f = ctypes.CDLL(lib).walk
    f.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_int, ctypes.c_int, ctypes.c_float,
                  ctypes.POINTER(ctypes.c_float)]
    f.restype = ctypes.c_int

    def call(scores, lift, per=4):
        n = len(scores)
        s, w = (ctypes.c_float * n)(*scores), (ctypes.c_float * n)()
        passes = f(s, n, per, lift, w)
        return passes, list(s), list(w)

    return call


LIFTS = range(-70, 101)
KMOVES = 8


def check(got, lift):
    """`got`: passes, the scores as binary32, their weights."""
    passes, s, w = got
    assert 1 <= passes <= KMOVES + 1, passes
    assert all(x + lift <= 15 for x in w)
    top = max(s)
    best = max(x for x, y in zip(w, s) if y == top)
    # the largest score's weight times the largest value scale is normal in
    # binary16: at most 9 under the centre, a move's rounding up to a whole
    # number, and half a step of a difference under 2^23
    assert best + lift >= 4 - 9 - 1 - 0.5
    # Weights are 2^(differences of scores).  From 2^23 on all numbers here are
    # whole, so that a move is exact and a weight's sum is rounded only where it
    # is as large as the difference; below, six moves and their rounding of
    # earlier weights, and one sum, each half a step of at most 2 |score| + 100,
    # of both keys.  What is over the highest weight is cut, which leaves 2^19.
    most = max(abs(y) for y in s)
    slack = 0.0 if most >= 2.0 ** 23 else 14 * (2 * most + 100) * 2.0 ** -24
    for x, y in zip(w, s):
        gap = top - y
        if gap > 0:
            assert best - x >= min(gap * (1 - 2.0 ** -22) - slack, 19)


@pytest.mark.parametrize("sign", [1, -1])
def test_one_key(walk, sign):
    for lift in LIFTS:
        for e in range(-10, 127):
            for m in (1.0, 1.25, 1.9999):
                check(walk([sign * m * 2.0 ** e], lift), lift)


def test_the_scores_that_repeated_for_ever(walk):
    """Scores of [2^28, 2^29) with a largest value scale of 2^-16 to 2^-13, and
    of 2^28 and more with one of 2^16 to 2^20."""
    for lift in (-16, -15, -14, -13, 16, 17, 18, 19, 20):
        for i in range(200):
            check(walk([3e8 + 32 * i], lift), lift)
            check(walk([2.0 ** 28 + 32 * i, 2.0 ** 28 + 32 * i + 32], lift), lift)
            check(walk([2.0 ** 34 + 2048 * i], lift), lift)


@pytest.mark.parametrize("shape", ["rising", "falling", "mixed", "ties", "neighbours"])
def test_many_keys(walk, shape):
    r = random.Random(shape)
    for lift in LIFTS:
        for e in (0, 4, 8, 16, 22, 24, 26, 27, 28, 29, 30, 31, 33, 36, 40, 64, 100, 125):
            for sign in (1, -1):
                a = 2.0 ** e * r.uniform(0.5, 1)
                if shape == "neighbours":
                    # a few of binary32's steps apart
                    step = 2.0 ** (e - 24)
                    s = [sign * a + step * r.randrange(-8, 9) for _ in range(24)]
                elif shape == "ties":
                    s = [sign * a * r.choice([1, 1, 0.75, 0.5]) for _ in range(24)]
                else:
                    s = [sign * a * r.random() for _ in range(24)]
                    s = {"rising": sorted(s), "falling": sorted(s)[::-1], "mixed": s}[shape]
                check(walk(s, lift), lift)


def test_infinite_and_missing_scores_end(walk):
    inf = float("inf")
    for lift in LIFTS:
        for s in ([inf], [1.0, inf], [1.0, 2.0, 3.0, 4.0, inf, 5.0], [-inf, 1.0], [3e38, -3e38],
                  [-3e38] * 8 + [3e38] * 8):
            passes, _, _ = walk(s, lift)
            assert passes == -1 or 1 <= passes <= KMOVES + 1  # -1: a move by infinity
