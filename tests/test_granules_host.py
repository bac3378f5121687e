"""Copies of unaligned rows by 16-byte granules (csrc/gdn_granules.h): every byte read lies in the
tensor, and every element arrives, for all alignments, row strides and edges.  On the host."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

DRIVER = r"""
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <vector>

#include "gdn_granules.h"

constexpr int CW = 64;  // channels of a tile

template <typename E, int LPR>
long check(int shift, int T, int C, int stride) {
    constexpr int PITCH = CW * (int)sizeof(E) + 16;
    const int64_t n = ((int64_t)(T - 1) * stride + C) * (int64_t)sizeof(E);
    // the tensor within guard bytes, `shift` bytes off a granule's start
    std::vector<uint8_t> all(n + 64 + 16);
    uint8_t* granule = (uint8_t*)(((uintptr_t)all.data() + 31) & ~(uintptr_t)15);
    uint8_t* lo = granule + shift;
    for (int64_t i = 0; i < n; ++i) lo[i] = (uint8_t)(i * 37 + i / 251);
    long bad = 0;
    for (int t = 0; t < T; ++t)
        for (int c0 = 0; c0 < C; c0 += CW) {
            uint8_t tile[PITCH];
            memset(tile, 0, sizeof(tile));
            const uint8_t* row = lo + ((int64_t)t * stride + c0) * (int64_t)sizeof(E);
            const int bytes = (C - c0 < CW ? C - c0 : CW) * (int)sizeof(E);
            const uint8_t* from = (const uint8_t*)((uintptr_t)row & ~(uintptr_t)15);
            for (int lane = 0; lane < LPR; ++lane)
                gdn::copy_granules<E, LPR, (PITCH / 16 + LPR - 1) / LPR>(
                    (uintptr_t)row, (uintptr_t)row + bytes, (uintptr_t)lo, (uintptr_t)(lo + n), lane,
                    [&](int o, int b) {
                        if (b < 1 || b > 16 || o % 16 || o + 16 > PITCH || from + o < lo ||
                            from + o + b > lo + n) {
                            ++bad;
                            return;
                        }
                        memset(tile + o, 0, 16);
                        memcpy(tile + o, from + o, b);
                    },
                    [&](int o) {
                        if (from + o < lo || from + o + (int)sizeof(E) > lo + n) {
                            ++bad;
                            return;
                        }
                        memcpy(tile + o, from + o, sizeof(E));
                    });
            if (memcmp(tile + (row - from), row, bytes)) ++bad;
        }
    return bad;
}

template <typename E>
long all() {
    long bad = 0;
    const int widths[] = {1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 33, 60, 63, 64, 65, 66, 71, 127, 128, 130};
    for (int shift = 0; shift < 16; shift += (int)sizeof(E))
        for (int C : widths)
            for (int gap = 0; gap < 10; ++gap)
                for (int T = 1; T < 12; ++T)
                    bad += check<E, 2>(shift, T, C, C + gap) + check<E, 4>(shift, T, C, C + gap);
    return bad;
}

int main() {
    const long bad = all<uint16_t>() + all<float>();
    printf("%ld wrong\n", bad);
    return bad != 0;
}
"""


def test_every_byte_read_lies_in_the_tensor(tmp_path):
    src, exe = tmp_path / "granules.cpp", tmp_path / "granules"
    src.write_text(DRIVER)
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "linear_attention_12_b200", "csrc"), str(src), "-o",
                    str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "0 wrong", out.stdout + out.stderr
