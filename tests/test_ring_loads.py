"""Which loads of a ring of stages a block waits for before it ends (CPU).

A model of the stages' barriers as waits by parity see them, with csrc/hc_loads.h as the kernel
compiles it: a loader issues loads until a wait gives up, its steps go on without loads, and at the
end any of the last loads may still be in flight.  After the waits that the rule names nothing may be
in flight, and no wait may be for a load that was never issued.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include "hc_loads.h"

constexpr int S = 4;

struct Stage {
    long phase = 0;         // phases that have ended
    bool flight = false;    // a load is on its way; the phase ends when it lands
    bool passed(unsigned parity) const { return (phase & 1) != parity; }
    void land() { if (flight) flight = false, ++phase; }
};

// bad ends: loads left in flight, or waits that nothing would end
static long run(long steps, long gave_up, unsigned in_flight, bool by_steps) {
    Stage st[S];
    hc::RingLoads<S> loads;
    for (long i = 0; i < steps; ++i) {
        if (i >= gave_up) continue;
        st[i % S].land();   // the stage was free: its last load has long landed
        loads.issue();
        st[i % S].flight = true;
    }
    for (int s = 0; s < S; ++s)
        if (!(in_flight >> s & 1)) st[s].land();
    long bad = 0;
    auto wait = [&](int s, unsigned parity) {
        if (st[s].passed(parity)) return;
        if (!st[s].flight) ++bad;
        st[s].land();
    };
    if (by_steps)           // the last S steps instead of the last S loads
        for (long i = steps > S ? steps - S : 0; i < steps; ++i)
            wait((int)(i % S), (unsigned)(i / S) & 1);
    else
        loads.in_flight(wait);
    for (int s = 0; s < S; ++s) bad += st[s].flight;
    return bad;
}

int main() {
    long bad[2] = {0, 0};
    for (int rule = 0; rule < 2; ++rule)
        for (long steps = 0; steps < 40; ++steps)
            for (long gave_up = 0; gave_up <= steps; ++gave_up)
                for (unsigned f = 0; f < 1u << S; ++f) bad[rule] += run(steps, gave_up, f, rule == 1);
    printf("%ld %ld\n", bad[0], bad[1]);
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_every_load_is_waited_for(tmp_path):
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "sinkhorn_mixing_gb300", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    loads, steps = map(int, subprocess.run([str(exe)], check=True, capture_output=True,
                                           text=True).stdout.split())
    assert loads == 0
    assert steps > 0        # the model tells the two rules apart
