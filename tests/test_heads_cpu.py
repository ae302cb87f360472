"""Addresses of heads as the kernels form them, on the host."""
import os
import shutil

import pytest

from test_q8_cpu import run_host

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")


def test_every_place_is_aligned(tmp_path):
    """The units that byte_bits allows divide the address of every place of a warp's step,
    those behind the heads too: a single head's stride, which may be odd, is not in them."""
    run_host(tmp_path, r"""
#include <cstdio>
#include "heads.h"
using namespace rmsn;
int main() {
    for (int es : {2, 4})
        for (long H : {1, 2, 5})
            for (long sh = 1; sh <= 70; ++sh)
                for (long row : {64, 66, 67, 420})
                    for (long T : {1, 3})
                        for (int n : {2, 3}) {
                            const int64_t st[] = {7 * row * 8, row * 8, sh};
                            const Heads x = heads((const void *)(uintptr_t)4096, st + 3 - n, n, es, H);
                            const uintptr_t bits = byte_bits(x, 1, T, H, es);
                            const unsigned unit = bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2;
                            bool ok = x.st == row * 8 && (H == 1 || x.head_bytes == (uint32_t)(sh * es)) && x.sh * es == x.head_bytes;
                            for (long t = 0; t < T; ++t)
                                for (uint32_t h = 0; h < 32; ++h)
                                    ok = ok && ((uintptr_t)x.p + t * x.st * es + (uint64_t)h * x.head_bytes) % unit == 0;
                            if (!ok) {
                                printf("es %d heads %ld stride %ld token stride %ld", es, H, sh, row * 8);
                                return 1;
                            }
                        }
    return 0;
}
""")
