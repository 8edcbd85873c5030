"""Where the routed experts' loads may read: every load of a pair of slabs,
past the last pair too, under both readings of the buffer address check (the
sum of the scalar and the lane's offset against the length; the lane's offset
against the unsigned 32-bit difference of the length and the scalar one)."""
import ctypes
import subprocess

import numpy as np
import pytest

from mixture_experts_layer_prefix_amd import _build


@pytest.fixture(scope="module")
def part_at(tmp_path_factory):
    """part_at() of csrc/parts.h as the host compiler makes it."""
    d = tmp_path_factory.mktemp("parts")
    src, lib = d / "parts.cpp", d / "parts.so"
    src.write_text('#include "parts.h"\nextern "C" uint32_t part_at(int i, int parts, uint32_t at, uint32_t n)'
                   " { return moe::part_at(i, parts, at, n); }\n")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", _build.CSRC, str(src), "-o", str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).part_at
    f.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_uint32, ctypes.c_uint32]
    f.restype = ctypes.c_uint32
    return f


def check(at, lanes, n, size):
    """No lane reads outside [0, n) under either reading."""
    assert at <= n
    lanes = np.asarray(lanes, np.int64)
    assert (at + lanes + size <= 1 << 32).all()      # the sum fits in 32 bits
    by_sum = at + lanes < n
    by_difference = lanes < (n - at) % (1 << 32)
    assert np.array_equal(by_sum, by_difference)
    assert (at + lanes[by_sum] + size <= n).all()    # whole or not at all


def issued(pairs):
    """Every pair that a wave asks for: its own, and those that it runs past the
    end with."""
    return sorted({i for wave in range(4) for i in range(wave, pairs + 9, 4)} | set(range(pairs + 7)))


SIZES = [128, 256, 384, 512, 640, 896, 1152, 1536, 2048, 7168, 7296]


@pytest.mark.parametrize("K", SIZES)
@pytest.mark.parametrize("rows", [1, 2, 17])
def test_tokens(part_at, K, rows):
    pairs = (K // 128 + 1) // 2
    quarter = np.arange(4) * 16
    for row in (0, rows - 1, None):                  # None: a lane without a token
        n, ns = rows * K, rows * (K // 32)
        o = row * K + quarter if row is not None else np.full(4, n)
        so = row * (K // 32) + np.arange(2) * 4 if row is not None else np.full(2, ns)
        for i in issued(pairs):
            for u in range(2):
                at = part_at(i, pairs, i * 256 + u * 128, n)
                check(at, np.concatenate([o, o + 64]), n, 16)
            check(part_at(i, pairs, i * 8, ns), so, ns, 4)


@pytest.mark.parametrize("K", SIZES)
def test_one_tokens_row(part_at, K):
    """The down projection by token: a row of h by itself, 256 bytes a load."""
    pairs = (K // 128 + 1) // 2
    for i in issued(pairs):
        check(part_at(i, pairs, i * 256, K), np.arange(16) * 16, K, 16)
        check(part_at(i, pairs, i * 8, K // 32), np.arange(2) * 4, K // 32, 4)


@pytest.mark.parametrize("K", SIZES)
@pytest.mark.parametrize("rows,all_rows", [(16, 128), (32, 256), (64, 128), (64, 1024)])
def test_weights(part_at, K, rows, all_rows):
    slabs = K // 128
    pairs = (slabs + 1) // 2
    n = rows * (K // 2)
    lane = np.arange(64)
    line = (lane >> 3) * (K // 2) + (lane & 7) * 16
    for i in issued(pairs):
        for q in range(rows // 8):
            check(part_at(i, pairs, i * 128 + q * 4 * K, n), line, n, 16)
    step = all_rows * 4
    for row in (0, rows, all_rows - rows):
        n = step * slabs - row * 4
        lanes = (lane % rows * 4 + lane // rows * step)[:2 * rows]
        for i in issued(pairs):
            for v in range(2 if rows == 64 else 1):
                check(part_at(2 * i + v, slabs, (2 * i + v) * step, n), lanes, n, 4)
