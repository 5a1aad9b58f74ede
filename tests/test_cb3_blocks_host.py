"""The 16-byte copies of 3-bit rows (csrc/cb3_blocks.h) on the host, over every row width,
place and step: sources on 16-byte boundaries and inside the array, also where a row has
ended and nothing is read; no byte past a row's end; every word of a step copied."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_routed_b200", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include "cb3_blocks.h"

int main() {
    long wrong[4] = {0, 0, 0, 0};
    for (uint32_t k = 32; k <= 4352; k += 32) {
        const uint32_t row_bytes = (k + 9) / 10 * 4, rw = row_bytes / 4, steps = (k + 127) / 128;
        for (uint32_t r = 0; r < 8; r++)        // rows of a block of 8, which starts on a boundary
            for (uint32_t j = 0; j < steps; j++) {
                const long row = (long)r * row_bytes;
                const uint32_t first = 128u * j / 10u, place = (r * rw + first) & 3u;
                const uint32_t last = (128u * j + 127u < k ? 128u * j + 127u : k - 1u) / 10u;
                uint32_t got = 0;                // words of the step, from its first
                for (uint32_t b = 0; b < (place == 3u ? 5u : 4u); b++) {
                    const moe::Cb3Block c = moe::cb3_block(r * rw, j, b, row_bytes);
                    if ((row + c.at) % 16) wrong[0]++;
                    if (row + c.at < 0 || c.bytes > 16) wrong[1]++;
                    if (c.bytes && c.at + (long)c.bytes > (long)row_bytes) wrong[2]++;
                    if (c.bytes && (c.at + 4 * (int)place) / 4 != (int)(first + 4 * b)) wrong[3]++;
                    for (uint32_t w = 0; 4 * w < c.bytes; w++) {
                        const int word = c.at / 4 + (int)w - (int)first;
                        if (word >= 0 && word < 14) got |= 1u << word;
                    }
                }
                for (uint32_t w = first; w <= last; w++)
                    if (!(got >> (w - first) & 1u)) wrong[3]++;
            }
    }
    printf("%ld %ld %ld %ld\n", wrong[0], wrong[1], wrong[2], wrong[3]);
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_sources_aligned_in_bounds_and_complete(tmp_path):
    src, exe = tmp_path / "blocks.cpp", tmp_path / "blocks"
    src.write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", CSRC, str(src), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0
    unaligned, outside, past_end, missing = map(int, out.stdout.split())
    assert (unaligned, outside, past_end, missing) == (0, 0, 0, 0)
