"""The shape rule of lora_bgmv_layer's pass over W (layer_shape.h), compiled for the host and looked over at
many sizes: tiles and shares cover the batch, everything fits, and no set of CTAs that fits an SM can ask
for more tensor memory than it has while it waits for the other CTAs of its clusters."""
import collections
import ctypes
import os
import subprocess

import pytest

import heterogeneous_adapters_sgmv_b200 as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(os.path.dirname(L.__file__), "csrc")

SRC = r"""
#include "layer_shape.h"
extern "C" void shape(int T, int h, int o, int n_sms, const int *of, int adapters, int *out)
{
    const lora::ClusterFit fit = {{of[0], of[1], of[2], of[3]}};
    const lora::StreamShape s = lora::stream_shape(T, h, o, n_sms, fit, adapters != 0);
    const int v[] = {s.N, s.NT, s.S, s.E, s.ctas, s.stages, s.share, s.ncols, s.recv, s.alias, s.smem};
    for (int i = 0; i < 11; ++i) out[i] = v[i];
}
"""
Shape = collections.namedtuple("Shape", "N NT S E ctas stages share ncols recv alias smem")
FIT = (148, 74, 33, 15)   # clusters of 1, 2, 4 and 8 CTAs that a B200 runs at once


@pytest.fixture(scope="module")
def shape(tmp_path_factory):
    d = tmp_path_factory.mktemp("shape")
    (d / "shape.cpp").write_text(SRC)
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wno-unused-function", "-I", CSRC, "-I",
                           os.path.join(ROOT, "include"), str(d / "shape.cpp"), "-o", str(d / "shape.so")])
    lib = ctypes.CDLL(str(d / "shape.so"))

    def call(T, h, o, adapters=True, fit=FIT):
        out = (ctypes.c_int * 11)()
        lib.shape(T, h, o, fit[0], (ctypes.c_int * 4)(*fit), int(adapters), out)
        return Shape(*out)

    return call


def sizes():
    for adapters in (True, False):
        for T in (1, 2, 16, 17, 32, 33, 48, 64, 65, 81, 96, 112, 128, 129, 161, 176, 192, 255, 256, 257, 300, 512, 777,
                  1030):
            for h in (8, 72, 128, 256, 512, 640, 1024, 1096, 4096, 14336):
                for tiles in (1, 2, 8, 15, 16, 17, 32, 33, 34, 74, 75, 112, 148, 149):
                    yield T, h, tiles * 128, adapters


def test_shape_covers_and_fits(shape):
    for T, h, o, adapters in sizes():
        s, what = shape(T, h, o, adapters), (T, h, o, adapters)
        assert s.N % 16 == 0 and 16 <= s.N <= 256 and (s.NT - 1) * s.N < T <= s.NT * s.N, what
        assert s.share * s.S >= min(s.N, T) and s.share % 4 == 0, what
        assert 1 <= s.stages <= 8 and s.smem <= 227 * 1024, what
        parts = s.E // 4
        per = -(-(s.share // parts) // 4) * 4
        assert parts * per >= s.share and s.N + parts * per <= s.ncols <= 512 // s.ctas, what
        recv = (s.S - 1) * s.share * 512
        ring = s.stages * (16384 + s.N * 128)
        if s.alias:
            assert s.recv == 0 and recv <= ring, what
        else:
            assert s.recv >= ring and s.recv % 16 == 0 and s.recv + recv + 1024 <= s.smem, what


def test_clusters_never_wait_for_each_others_tensor_memory(shape):
    """Every CTA of a cluster that fits an SM has its columns, so none can hold some while it waits for a peer
    that waits for more: over all sets of such CTAs, also of other launches, columns stay within 512."""
    kinds = {(97 * 1024, 64)}   # the long segments' shrink
    for T, h, o, adapters in sizes():
        s = shape(T, h, o, adapters)
        if s.S > 1:
            kinds.add((s.smem, s.ncols))
    # the smallest of each number of columns fill an SM worst
    least = {}
    for smem, cols in kinds:
        least[cols] = min(smem, least.get(cols, smem))

    def worst(room):
        return max([0] + [cols + worst(room - smem - 1024) for cols, smem in least.items() if smem + 1024 <= room])

    assert worst(228 * 1024) <= 512


def test_gpu_sizes_reach_the_forms_they_are_for(shape):
    """The sizes of test_bgmv_layer_long_rings, with and without ids."""
    from tests.test_gpu_layer_forms import ROUNDS
    seen, parts = set(), set()
    for T, h, o in ROUNDS:
        s = shape(T, h, o)
        if -(-h // 64) // s.S > 2 * s.stages:
            seen.add((s.S, s.ctas, bool(s.alias)))
        if T > 1:
            parts.add(min(4, max(1, h // 1024)) if T <= 512 else 1)
    assert {(1, 1, False), (1, 2, False), (2, 1, False), (4, 1, False), (8, 1, False), (2, 1, True), (2, 2, True),
            (4, 2, True), (8, 2, True), (8, 2, False)} <= seen
    assert parts == {1, 2, 3, 4}
