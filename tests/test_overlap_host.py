"""The refusal of outputs that overlap inputs or one another (ttt_overlap.h), compiled for the host:
every pair of ranges at and around its ends against sets of bytes."""
import ctypes
import itertools
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def clash(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("emu") / "overlap_emu.so")
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC",
                    os.path.join(HERE, "host_emu", "overlap_emu.cpp"), "-o", so], check=True)
    f = ctypes.CDLL(so).overlap_host_run

    def call(*ranges):
        flat = [x for r in ranges for x in r]
        return bool(f((ctypes.c_ulonglong * len(flat))(*flat)))
    return call


FAR = [(10 ** 6 * i, 64) for i in range(1, 6)]


def test_ranges_apart_pass(clash):
    assert not clash(*FAR)
    assert not clash((0, 64), (0, 64), *FAR[2:])               # arrays that are not there
    assert not clash((4096, 64), (4160, 64), (4032, 64), (4224, 64), (1 << 62, 1 << 40))  # neighbours


def test_pairs_against_sets_of_bytes(clash):
    for a, n, b, m in itertools.product(range(100, 106), range(4), range(100, 106), range(4)):
        meet = bool(set(range(a, a + n)) & set(range(b, b + m)))
        for i, j in itertools.combinations(range(5), 2):
            r = list(FAR)
            r[i], r[j] = (a, n), (b, m)
            want = meet and i < 2                             # two inputs may share memory
            if (i, j) == (0, 3) and (a, n) == (b, m):
                want = False                                  # the first output over its input
            assert clash(*r) == want, (i, j, a, n, b, m)


def test_sizes_past_32_bits(clash):
    r = list(FAR)
    r[0], r[4] = (1 << 40, 1 << 36), ((1 << 40) + (1 << 36) - 1, 1)
    assert clash(*r)
    r[4] = ((1 << 40) + (1 << 36), 1)
    assert not clash(*r)
