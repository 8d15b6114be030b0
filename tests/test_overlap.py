"""Whether two arrays of rows share a byte (csrc/overlap.h), against a look at every byte, and the calls
of moe_linear that it refuses."""
import subprocess

import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe
from quantized_routed_expert_moe_gb300 import build
from test_decoder_ops_host import P
from test_prefill_ops_host import linear_desc

PROGRAM = r"""
#include <cstdio>
#include <cstring>
#include "overlap.h"

static char room[4096];

static bool by_bytes(moe::Span a, moe::Span b) {
    static unsigned char seen[4096];
    std::memset(seen, 0, sizeof seen);
    for (int64_t i = 0; i < a.rows; ++i)
        for (int64_t k = 0; k < a.width; ++k) seen[(const char*)a.at - room + i * a.pitch + k] = 1;
    for (int64_t i = 0; i < b.rows; ++i)
        for (int64_t k = 0; k < b.width; ++k)
            if (seen[(const char*)b.at - room + i * b.pitch + k]) return true;
    return false;
}

int main() {
    unsigned state = 1;
    auto draw = [&](int n) { return (int)((state = state * 1664525u + 1013904223u) >> 8) % n; };
    int met = 0;
    for (int n = 0; n < 400000; ++n) {
        auto span = [&] {
            const int64_t rows = 1 + draw(6), width = 1 + draw(12), pitch = width + (draw(3) ? draw(14) : 0);
            return moe::Span{room + draw(120), rows, width, pitch};
        };
        moe::Span a = span(), b = span();
        if (draw(2) && b.width <= a.pitch) b.pitch = a.pitch;   // columns of one buffer
        const bool want = by_bytes(a, b);
        met += want;
        if (moe::overlap(a, b) != want || moe::overlap(b, a) != want) {
            std::printf("%ld: %ld x %ld / %ld; %ld: %ld x %ld / %ld\n", (long)((char*)a.at - room), (long)a.rows, (long)a.width,
                        (long)a.pitch, (long)((char*)b.at - room), (long)b.rows, (long)b.width, (long)b.pitch);
            return 1;
        }
    }
    if (met < 1000 || met > 399000) return 2;
    if (moe::overlap({nullptr, 4, 4, 4}, {room, 4, 4, 4}) || moe::overlap({room, 0, 4, 4}, {room, 4, 4, 4})) return 3;
    return 0;
}
"""


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_overlap_against_a_look_at_every_byte(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], timeout=60, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def status(d, x, w, bias, residual, y, T):
    """Of a call on a device that is not there: nothing is ever launched."""
    import ctypes
    return moe.lib().moe_linear(ctypes.byref(d), x, w, bias, residual, y, T, 1000, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="test_gpu_overlaps.py makes such calls, with memory")
def test_a_linear_that_would_overwrite_its_inputs_is_refused():
    far = P + (1 << 20)
    same = linear_desc(in_features=64, out_features=64, y_stride=64, residual_stride=64)
    INVALID = 1
    assert status(same, P, far, None, None, P, 3) == INVALID            # y is x
    assert status(same, far, P, None, None, P, 3) == INVALID            # y is w
    assert status(same, far, P, None, None, P + 2 * 64 * 63, 3) == INVALID   # y on w's last row
    assert status(same, far, P, None, None, P + 2 * 64 * 64, 3) != INVALID   # y behind it
    assert status(same, far, far + 65536, P + 128, None, P, 3) == INVALID    # bias in y
    assert status(same, far, far + 65536, None, P + 128, P, 3) == INVALID    # residual a row later
    # columns of one buffer: x in 0..63, y in 64..127 or 56..119
    d = linear_desc(in_features=64, out_features=64, x_stride=192, y_stride=192, residual_stride=192)
    assert status(d, P, far, None, None, P + 2 * 64, 3) != INVALID
    assert status(d, P, far, None, None, P + 2 * 56, 3) == INVALID
    # in place on the residual, and the residual's columns beside y's
    assert status(d, far, far + 65536, None, P, P, 3) != INVALID
    assert status(d, far, far + 65536, None, P + 2 * 64, P, 3) != INVALID
