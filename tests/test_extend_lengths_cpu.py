"""The extend kernel's arithmetic on lengths, up to 2^31 - 1 positions: its own functions, compiled for the CPU with
32-bit arithmetic that wraps, against integers that do not."""
import ctypes
import os
import random
import re
import subprocess

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_gqa_decode_hpc_gb300", "csrc",
                   "prefill_kernel.cu")
TOP = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    with open(SRC) as f:
        text = f.read()
    names = ("tile_kv", "keys_seen")
    bodies = [re.search(r"__device__ __forceinline__ int %s\(.*?\n}\n" % n, text, re.S).group(0) for n in names]
    last = re.search(r"if \((kv0.*?lim.*?)\) \{", text).group(1)
    code = "constexpr int kExtendTileTokens = 16;\n" + "".join(
        b.replace("__device__ __forceinline__", 'extern "C"') for b in bodies)
    code += 'extern "C" int reaches_past(int kv0, int lim) { return %s; }\n' % last
    d = tmp_path_factory.mktemp("lengths")
    (d / "x.cpp").write_text(code)
    subprocess.run(["g++", "-O1", "-fwrapv", "-shared", "-fPIC", str(d / "x.cpp"), "-o", str(d / "x.so")], check=True)
    return ctypes.CDLL(str(d / "x.so"))


def cases():
    rng = random.Random(1)
    for L in [1, 15, 16, 17, 63, 64, 65, 1000, 134217728, TOP - 128, TOP - 64, TOP - 63, TOP - 62, TOP - 16, TOP - 1, TOP]:
        for n in {1, 2, 15, 16, 17, 33, 1000, rng.randint(1, 100000)}:
            if n <= L:
                for t0 in {0, 16, n // 16 * 16, (n - 1) // 16 * 16}:
                    yield L, n, t0


def test_tiles_and_limits_of_all_lengths(lib):
    for L, n, t0 in cases():
        want = 0 if t0 >= n else -(-min(L, L - n + t0 + 16) // 64)
        assert lib.tile_kv(L, n, t0) == want, (L, n, t0)
        for tok in range(t0, t0 + 32):
            assert lib.keys_seen(L, n, tok) == min(L, L - n + 1 + tok)
        seen = min(L, L - n + 1 + min(t0, n - 1))
        for j in {0, max(0, want - 2), max(0, want - 1)}:  # the last tiles hide what lies past the row's limit
            assert bool(lib.reaches_past(64 * j, seen)) == (64 * j + 64 > seen), (L, n, t0, j)
