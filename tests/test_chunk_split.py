"""The split of chunk attention over the GPU against brute force on the CPU: csrc/chunk_attn.cuh
compiled for the host (tests/chunk_split.cu). Every step of every unit is taken once, in order;
a cut unit's parts lie in the runs that the join reads; no run is longer than the others' plus a
step and a unit's start."""
import ctypes
import os
import random
import subprocess

import pytest

from block_sparse_linear_b200 import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("split") / "chunk_split.so")
    subprocess.run([build.NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-O2", "-std=c++17",
                    "-shared", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
                    "-I", os.path.join(build.ROOT, "include"), "-I", os.path.join(build.HERE, "csrc"),
                    os.path.join(HERE, "chunk_split.cu"), "-o", so], check=True)
    lib = ctypes.CDLL(so)

    def call(f32, d, hkv, group, block, max_new, lens, n_new, mbp=None):
        arr = ctypes.c_int32 * len(lens)
        mbp = mbp or max(1, -(-max(lens) // block))
        longest = ctypes.c_int64()
        line = lib.chunk_split_check(f32, d, len(lens), hkv, group, block, mbp, max_new, arr(*lens),
                                     arr(*n_new), ctypes.byref(longest))
        assert line == 0, f"chunk_split.cu:{line} f32={f32} d={d} hkv={hkv} group={group} " \
                          f"block={block} max_new={max_new} lens={lens[:40]} n_new={n_new[:40]}"
        return longest.value

    return call


def log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


@pytest.mark.parametrize("seed", range(8))
def test_random_batches(check, seed):
    rng = random.Random(seed)
    for _ in range(1500):
        batch = log_int(rng, 1, 3000 if rng.random() < 0.2 else 200)
        top = log_int(rng, 1, min(1 << 20, max(4, (1 << 24) // batch)))
        max_new = rng.choice((1, log_int(rng, 1, 64), log_int(rng, 1, 3000)))
        low = log_int(rng, 1, top)
        lens = [rng.randint(low, top) for _ in range(batch)]
        empty = rng.choice((0.0, 0.2, 0.9))
        n_new = [0 if rng.random() < empty else rng.randint(0, min(n, max_new)) for n in lens]
        if rng.random() < 0.1:                          # out of range: no part in the split
            n_new[rng.randrange(batch)] = rng.choice((-1, max_new + 1))
        check(rng.randint(0, 1), rng.choice((64, 128)), rng.choice((1, 2, 3, 8)),
              rng.choice((1, 2, 4)), rng.choice((64, 128)), max_new, lens, n_new)


@pytest.mark.parametrize("f32", [0, 1])
@pytest.mark.parametrize("d,block", [(64, 64), (128, 128)])
def test_largest_and_smallest(check, f32, d, block):
    top = 32768 * block                                 # the longest block table
    for group in (1, 2, 4):
        for n in (1, 2, 128 // group, 128 // group + 1, 256 // group, 5000, top):
            check(f32, d, 1, group, block, n, [top], [n])
            check(f32, d, 8, group, block, n, [top, n, top - 1, n + 1], [n, n, 0, n])
        check(f32, d, 4, group, block, 1, [top] * 300, [1] * 300)
        check(f32, d, 1, group, block, 1, [1] * (1 << 17), [1] * (1 << 17))
        check(f32, d, 32, group, block, 3, [7, 300] * (1 << 14), [3, 0] * (1 << 14))
        check(f32, d, 2, group, block, 1, [5, 9], [0, 0])
    # as many (sequence, KV head) pairs as there may be, each as long as there is: the costs'
    # sum stays below the units' count beside it
    batch = 1 << 14
    check(f32, d, 256, 1, block, 1, [top] * batch, [1] * batch)


def test_whole_runs_of_equal_units(check):
    """Batches around the number of runs and of steps where the rules on starts change."""
    for f32 in (0, 1):
        for batch in (1, 37, 74, 147, 148, 149, 296, 383, 384, 385, 768, 769):
            for L in (1, 63, 64, 65, 127, 128, 129, 1024, 2048, 2049, 16 * 128, 17 * 128):
                for hkv in (1, 4):
                    check(f32, 64, hkv, 2, 64, 1, [L] * batch, [1] * batch)
                    check(f32, 128, hkv, 4, 64, 70, [L] * batch, [min(L, 70)] * batch)
