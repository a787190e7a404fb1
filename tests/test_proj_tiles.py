"""How the products behind la_linear_* are cut (csrc/linear_cut.hpp, compiled here for the host): the shapes that the
GPU tests run reach every kernel, with one round of workgroups and with more, whole sums and cut ones."""
import ctypes
import os
import subprocess

import pytest

from tests.proj_tiles import DEEP, FEW, FORWARD, GRADIENTS, SLOTS, T64, T128, T256

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_state_qat_amd", "csrc")
SOURCE = """
#include "linear_cut.hpp"
using namespace la;
extern "C" void forward(int M, int N, int K, int64_t* out) {
    if (M <= few_tokens(N, K)) { out[0] = -1, out[1] = 1, out[2] = (N + 15) / 16; return; }
    const Cut c = cut_forward(M, N, K);
    out[0] = c.tiling, out[1] = c.parts, out[2] = gemm_units_of(c.tiling, N, M, c.parts);
}
extern "C" void gradients(int M, int N, int K, int64_t* out) {
    const GradientCuts c = cut_gradients(M, N, K);
    out[0] = c.dx.tiling, out[1] = c.dx.parts, out[2] = gemm_units_of(c.dx.tiling, K, M, c.dx.parts);
    out[3] = c.dw.tiling, out[4] = c.dw.parts, out[5] = gemm_units_of(c.dw.tiling, K, N, c.dw.parts);
    out[6] = c.pair;
}
"""


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    at = tmp_path_factory.mktemp("cut")
    (at / "cut.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++20", "-O2", "-ffp-contract=off", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(at / "cut.cpp"),
                    "-o", str(at / "cut.so")], check=True)
    lib = ctypes.CDLL(str(at / "cut.so"))

    def call(which, M, N, K):
        out = (ctypes.c_int64 * 7)()
        getattr(lib, which)(M, N, K, out)
        return list(out)

    return call


@pytest.mark.parametrize("M,N,K,tiles,rounds", FORWARD)
def test_forward(cut, M, N, K, tiles, rounds):
    got, parts, units = cut("forward", M, N, K)[:3]
    assert got == tiles and parts == 1 and (units > SLOTS.get(got, units)) == rounds


@pytest.mark.parametrize("M,N,K,dx,dw,pair", GRADIENTS)
def test_gradients(cut, M, N, K, dx, dw, pair):
    out = cut("gradients", M, N, K)
    for at, (tiles, parts, rounds) in ((0, dx), (3, dw)):
        assert (out[at], out[at + 1], out[at + 2] > SLOTS[out[at]]) == (tiles, parts, rounds)
    assert bool(out[6]) == pair


def test_every_kernel_is_among_them():
    assert {(c[3], c[4]) for c in FORWARD} == {(FEW, False)} | {(t, r) for t in (DEEP, T64, T128, T256) for r in (False, True)}
    alone = {(t, parts > 1, r) for c in GRADIENTS if not c[5] for t, parts, r in c[3:5]}
    assert alone >= {(t, False, r) for t in (DEEP, T64, T128, T256) for r in (False, True)}
    assert alone >= {(t, True, False) for t in (DEEP, T64, T128, T256)} | {(t, True, True) for t in (T64, T128, T256)}
    assert {c[3][0] for c in GRADIENTS if c[5]} == {DEEP, T64, T128}
    assert {K % 128 // 16 for _, _, K, *_ in FORWARD} >= {0, 1, 2, 3, 5, 7} and any(-(-K // 128) > 8 for _, _, K, *_ in FORWARD)
