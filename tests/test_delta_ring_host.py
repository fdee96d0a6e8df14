"""The thread that fills a ring of stages in the gated delta rule's scans (ttt_delta_ring.cuh), on the
host (tests/host_emu/delta_ring_emu.cpp): whatever the number of steps, and wherever the consumer
gives up, no copy is in flight when the thread is gone, since the block's shared memory may go with
it. A consumer that gives up when the last copies have been issued leaves nobody else to wait."""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "host_emu", "delta_ring_emu.cpp")


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("emu") / "delta_ring_emu.so")
    subprocess.run(["g++", "-std=c++20", "-O2", "-shared", "-fPIC", SRC, "-o", so], check=True)
    L = ctypes.CDLL(so)
    L.delta_ring_host_run.restype = ctypes.c_int
    L.delta_ring_host_run.argtypes = [ctypes.c_int] * 4 + [ctypes.POINTER(ctypes.c_int)]

    def call(stages, steps, latency, give_up):
        done = ctypes.c_int()
        return L.delta_ring_host_run(stages, steps, latency, give_up, done), done.value
    return call


@pytest.mark.parametrize("stages", [1, 2, 3, 4])
@pytest.mark.parametrize("latency", [0, 1, 17])
def test_no_copy_outlives_the_filling_thread(run, stages, latency):
    for steps in range(12):
        assert run(stages, steps, latency, -1) == (0, steps)
        for give_up in range(steps + 1):
            flying, done = run(stages, steps, latency, give_up)
            assert flying == 0 and done == min(steps, give_up + stages), (steps, give_up)
