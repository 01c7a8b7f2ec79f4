"""The rule by which a kernel's waits are recorded and given up, and the account of a ring's copies
(csrc/wait_rule.cuh), run on the host with phases that complete after so many polls, or never."""
from __future__ import annotations

import subprocess

import pytest

from rank_state_read_b200 import build as rbuild

HEAD = r"""
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include "wait_rule.cuh"
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); std::exit(1); } } while (0)
"""

WAITS = r"""
struct Cta { int limit = 0, polls = 0, late = 0, stops = 0; bool stop = false; };
struct Ops {
    Cta &c;
    int after;  // polls until the phase completes; negative: never
    int limit() const { return c.stop ? -1 : c.limit; }
    bool stopped() const { return c.stop; }
    bool test() const { return after == 0; }
    bool poll() { ++c.polls; return after > 0 && --after == 0; }
    void late() { ++c.late; }
    void stop() { c.stop = true; ++c.stops; }
};
int main()
{
    for (int limit : {0, 1, 7}) {
        for (int most : {1, 50}) {
            Cta c{limit};
            CHECK(sk::wait_by_rule(Ops{c, 0}, most) && c.polls == 0 && c.late == 0);
            if (limit) CHECK(sk::wait_by_rule(Ops{c, limit}, most) && c.late == 0);  // in time
            // late, but it comes: recorded, and the wait goes on for it
            Cta d{limit};
            CHECK(sk::wait_by_rule(Ops{d, limit + most}, most) && d.late == most && !d.stop);
            // it never comes: given up after limit + most polls
            Cta e{limit};
            CHECK(!sk::wait_by_rule(Ops{e, -1}, most) && e.stop && e.stops == 1);
            CHECK(e.polls == limit + most);
            // and then no wait that begins polls, however many there are: each looks once
            for (int i = 0; i < 100000; ++i) {
                CHECK(!sk::wait_by_rule(Ops{e, -1}, most));
                CHECK(!sk::wait_by_rule(Ops{e, 3}, most));
                CHECK(sk::wait_by_rule(Ops{e, 0}, most));
            }
            CHECK(e.polls == limit + most);
            // a wait that had begun when another one was given up ends within its own limit
            struct Other : Ops {
                bool poll() { if (++c.polls == 1) c.stop = true; return false; }
            };
            Cta f{limit};
            CHECK(!sk::wait_by_rule(Other{{f, -1}}, most) && f.polls == (limit > 1 ? limit : 1));
        }
    }
    return 0;
}
"""

RING = r"""
#include <random>
// barriers as the hardware counts them: `done` completed phases a stage, a test of parity p succeeds when the
// phase that is open has the other one
int main()
{
    std::mt19937 g(1);
    for (int run = 0; run < 20000; ++run) {
        const int stages = 1 + g() % 5, items = 1 + g() % 20, lose = g() % (items + 1);
        sk::RingPhases r;
        int done[16] = {}, out[16] = {};  // completed phases, copies asked for
        bool skipped[64];
        for (int i = 0; i < items; ++i) skipped[i] = g() % 4 == 0;  // rows to leave alone bring nothing
        auto bring = [&](int i) { if (!skipped[i]) { r.issued(i % stages); ++out[i % stages]; } };
        auto test = [&](int st) { return (unsigned)(done[st] & 1) != r.parity(st); };
        for (int i = 0; i < stages && i < items; ++i) bring(i);
        for (int i = 0; i < items; ++i) {
            const int st = i % stages;
            if (!skipped[i]) {
                CHECK(r.pending(st) && !test(st));  // it has not landed: a wait waits
                if (i == lose) break;               // given up: neither landed() nor the next copy
                ++done[st];
                CHECK(test(st));
                r.landed(st);
            }
            if (i + stages < items) bring(i + stages);
        }
        // what is under way is what was asked for and has not landed, and a wait for it waits for that copy
        for (int st = 0; st < stages; ++st) {
            CHECK(r.pending(st) == (out[st] > done[st]) && out[st] - done[st] <= 1);
            if (r.pending(st)) {
                CHECK(!test(st));
                ++done[st];
                CHECK(test(st));
            }
        }
    }
    return 0;
}
"""


def run(tmp_path, source):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(HEAD + source)
    subprocess.run(["g++", "-std=c++17", "-x", "c++", "-I", rbuild.CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("source", [WAITS, RING], ids=["waits", "ring"])
def test_rule(tmp_path, source):
    run(tmp_path, source)
