"""The barriers of a ring of copies after a kernel has given up: each phase ends when, and only when, every copy issued for it has landed.

The accounting is compiled for the host and run against a model of the barriers, over producers that stopped at any use.
"""
import ctypes
import itertools
import os
import random
import subprocess

import pytest

STAGES, PIECE = 4, (16384, 32768)  # bytes of one SM's piece of A and of B
SOURCE = r"""
#include "ct_settle.h"
extern "C" void owed(unsigned k, unsigned first, unsigned second, int pair, unsigned bytes, unsigned* out) {
    const ct::Owed o = ct::owed(k, first, second, pair != 0, bytes);
    out[0] = o.arrive;
    out[1] = o.announce;
    out[2] = o.absent;
}
extern "C" unsigned unsettled_from(unsigned n, unsigned stages) { return ct::unsettled_from(n, stages); }
"""


@pytest.fixture(scope="module")
def settle(tmp_path_factory, repo_root):
    d = tmp_path_factory.mktemp("settle")
    (d / "settle.cpp").write_text(SOURCE)
    csrc = os.path.join(repo_root, "transposed_convolution_convtranspose1_gb300", "csrc")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I", csrc, "-o", str(d / "settle.so"), str(d / "settle.cpp")])
    return ctypes.CDLL(str(d / "settle.so"))


class Barrier:
    """Two arrivals a phase, and as many bytes landed as announced."""

    def __init__(self):
        self.pending, self.bytes, self.ended = 2, 0, False

    def check(self):
        assert not self.ended or (self.pending, self.bytes) == (0, 0), "something came after the phase's end"
        self.ended = self.ended or (self.pending == 0 and self.bytes == 0)

    def arrive(self, announced):
        assert self.pending > 0, "one arrival too many"
        self.bytes += announced
        self.pending -= 1
        self.check()

    def land(self, n):
        self.bytes -= n
        self.check()


def run(settle, sms, counts, late, rng, mend=True):
    """counts[operand][SM]: uses issued.  Copies land at random, `late` of them after the accounting.  Whether every phase ended."""
    n = max(c for per_sm in counts for c in per_sm)
    out = (ctypes.c_uint * 3)()
    ended = True
    for k in range(settle.unsettled_from(n, STAGES), n):
        bar = Barrier()
        copies = []
        for i in (0, 1):
            if counts[i][0] > k:
                bar.arrive(sms * PIECE[i])
            copies += [PIECE[i] for sm in range(sms) if counts[i][sm] > k]
        rng.shuffle(copies)
        early = copies[min(late, len(copies)):]
        for c in early:
            bar.land(c)
        if mend:
            for i in (0, 1):
                settle.owed(k, counts[i][0], counts[i][1] if sms == 2 else 0, int(sms == 2), PIECE[i], out)
                if out[0]:
                    bar.arrive(out[1])
                if out[2]:
                    bar.land(out[2])
        assert not bar.ended or late == 0 or not copies, "a phase ended before its copies had landed"
        for c in copies[:len(copies) - len(early)]:
            bar.land(c)
        ended = ended and bar.ended
    return ended


@pytest.mark.parametrize("sms", [1, 2])
def test_every_phase_ends_with_its_last_copy(settle, sms):
    rng = random.Random(sms)
    for base in (0, 3, 9):  # uses that have landed and been read
        for more in itertools.product(range(STAGES + 1), repeat=2 * sms):
            counts = [[base + more[i * sms + s] for s in range(sms)] for i in (0, 1)]
            for late in range(2 * sms + 1):
                assert run(settle, sms, counts, late, rng)


def test_it_takes_the_accounting():
    """Without it a phase whose producers stopped at different uses never ends, and none that all reached is touched."""
    class Plain:
        @staticmethod
        def unsettled_from(n, stages):
            return max(0, n - stages)
    rng = random.Random(3)
    assert not run(Plain, 2, [[3, 3], [3, 2]], 0, rng, mend=False)
    assert not run(Plain, 2, [[2, 3], [2, 3]], 0, rng, mend=False)
    assert run(Plain, 2, [[3, 3], [3, 3]], 0, rng, mend=False)
