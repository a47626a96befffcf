"""The latent ring of the paged kernels, simulated on the host against the
arithmetic that a CTA which gives up uses to wait for its copies in flight."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mla_latent_kv_07_gb300", "csrc")
PER = 4


@pytest.fixture(scope="module")
def last_load(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    src, so = str(d / "ring.cpp"), str(d / "ring.so")
    with open(src, "w") as f:
        f.write('#include "ring.cuh"\nextern "C" int last_load(const int* issued, int per, int slots, int s) {\n'
                "  return mla::paged::last_load(issued, per, slots, s);\n}\n")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", so, src], check=True)
    lib = ctypes.CDLL(so)

    def call(issued, slots, s):
        return lib.last_load((ctypes.c_int * PER)(*issued), PER, slots, s)

    return call


class Ring:
    """Producers load their pairs when the slot's load before has been read;
    loads land in any order; a tile is read pair by pair once it is complete."""

    def __init__(self, slots, tiles, rng):
        self.slots, self.tiles, self.rng = slots, tiles, rng
        self.issued, self.landed, self.read = [0] * PER, set(), 0
        self.made = []

    def flying(self):
        return [n for n in self.made if n not in self.landed]

    def step(self):
        moves = [("issue", m) for m in range(PER)
                 if self.issued[m] < self.tiles and PER * self.issued[m] + m - self.slots < self.read]
        moves += [("land", n) for n in self.flying()]
        if self.read in self.landed:
            moves.append(("read", 0))
        if not moves:
            return False
        what, x = self.rng.choice(moves)
        if what == "issue":
            self.made.append(PER * self.issued[x] + x)
            self.issued[x] += 1
        elif what == "land":
            self.landed.add(x)
        else:
            self.read += 1
        return True


@pytest.mark.parametrize("slots", [4, 8, 10])
def test_every_copy_in_flight_is_waited_for(last_load, slots):
    rng = random.Random(slots)
    only_newest_misses = 0
    for _ in range(400):
        r = Ring(slots, rng.randint(1, 12), rng)
        for _ in range(rng.randint(0, 200)):
            if not r.step():
                break
        last = [last_load(r.issued, slots, s) for s in range(slots)]
        for s, n in enumerate(last):
            mine = [x for x in r.made if x % slots == s]
            assert n == max(mine, default=-1)
            # a parity wait tells a phase from the next one only: all loads
            # before the last one have landed, and none follows
            assert all(x in r.landed for x in mine if x != n)
        assert set(r.flying()) <= set(last)
        newest = {PER * (i - 1) + m for m, i in enumerate(r.issued) if i}
        only_newest_misses += not set(r.flying()) <= newest
    # waiting for each producer's newest copy alone would leave others in
    # flight, unless a producer has one slot
    assert (only_newest_misses > 0) == (slots > PER)
