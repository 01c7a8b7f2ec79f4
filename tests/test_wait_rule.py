"""The rule by which a kernel's waits are recorded and given up (csrc/wait_rule.cuh), run on the host with
phases that complete after so many polls, or never."""
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


def run(tmp_path, source):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(HEAD + source)
    subprocess.run(["g++", "-std=c++17", "-x", "c++", "-I", rbuild.CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("source", [WAITS], ids=["waits"])
def test_rule(tmp_path, source):
    run(tmp_path, source)
