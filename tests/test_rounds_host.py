"""How loops on the GPU end whatever they find (csrc/rounds.h), without a GPU.  Warps that begin rounds of work together, as the
builders of ember_adapter_project's tiles do: whoever gives up, in whichever round and place, nobody is left waiting at the vote
(threads stand for the warps, a barrier with a time limit for the vote).  Walks along a line, as the CTAs of a shared prefix
make: places that nobody owns, which only arrays that change during the call can make, end them."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "gqa_transformer_decode_gb300", "csrc")
PROGRAM = r"""
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <thread>
#include <vector>

#include "rounds.h"

struct Vote {                    // of `count` workers; none may wait longer than two seconds
    std::mutex m;
    std::condition_variable cv;
    int count, here = 0, phase = 0;
    bool and_ = true, result = true;
    bool all(bool ok) {
        std::unique_lock<std::mutex> l(m);
        and_ = and_ && ok;
        const int mine = phase;
        if (++here == count) {
            result = and_;
            and_ = true;
            here = 0;
            ++phase;
            cv.notify_all();
            return result;
        }
        if (!cv.wait_for(l, std::chrono::seconds(2), [&] { return phase != mine; })) {
            std::printf("a worker was left waiting at the vote\n");
            std::fflush(stdout);
            std::_Exit(1);
        }
        return result;
    }
};

int main() {
    int runs = 0;
    for (int workers : {1, 4, 8})
        for (int rounds : {0, 1, 2, 5})
            for (int who = -1; who < workers; ++who)             // -1: nobody gives up
                for (int when = 0; when < (who < 0 ? 1 : rounds); ++when)
                    for (int in_work = 0; in_work < 2; ++in_work) {
                        Vote v;
                        v.count = workers;
                        std::vector<int> done(workers), result(workers);
                        std::vector<std::thread> ts;
                        for (int w = 0; w < workers; ++w)
                            ts.emplace_back([&, w] {
                                result[w] = ember::rounds_together(
                                    rounds, [&](int i) { return in_work || w != who || i != when; }, [&](bool ok) { return v.all(ok); },
                                    [&](int i) {
                                        ++done[w];
                                        return !in_work || w != who || i != when;
                                    });
                            });
                        for (auto& t : ts) t.join();
                        ++runs;
                        for (int w = 0; w < workers; ++w) {
                            // a round is begun by all or by none; who gave up says so, the others from the next vote on
                            const int want = who < 0 ? rounds : when + in_work;
                            const bool whole = who < 0 || (in_work && when + 1 == rounds && w != who);
                            if (done[w] != want || (result[w] != 0) != whole) {
                                std::printf("worker %d of %d: %d of %d rounds, %d\n", w, workers, done[w], rounds, result[w]);
                                return 1;
                            }
                        }
                    }
    std::printf("%d ways to end\n", runs);
    return 0;
}
"""


WALKS = r"""
#include <cstdio>

#include "rounds.h"

int main() {
    // steps from the place 3 of a line of 10, and where they lead (-1: the end)
    const struct { int steps[4], places[4]; } walks[] = {
        {{2, 1, 4, 9}, {5, 6, -1, 0}}, {{7, 0, 0, 0}, {-1, 0, 0, 0}}, {{6, 1, 0, 0}, {9, -1, 0, 0}}, {{100, 0, 0, 0}, {-1, 0, 0, 0}},
        {{0, 0, 0, 0}, {-1, 0, 0, 0}}, {{-1, 0, 0, 0}, {-1, 0, 0, 0}}, {{2, 0, 0, 0}, {5, -1, 0, 0}}, {{2147483647, 0, 0, 0}, {-1, 0, 0, 0}}};
    for (const auto& w : walks) {
        unsigned at = 3;
        for (int i = 0; i < 4; ++i) {
            const bool on = ember::walk_on(at, w.steps[i], 10);
            if (on != (w.places[i] >= 0) || (on && at != (unsigned)w.places[i])) return 1;
            if (!on) break;
        }
    }
    unsigned at = 4294967290u;                   // no sum beyond 32 bits
    return ember::walk_on(at, 5, 4294967295u) || !ember::walk_on(at, 4, 4294967295u) || at != 4294967294u;
}
"""


def run(tmp_path, program):
    src, exe = tmp_path / "rounds.cpp", tmp_path / "rounds"
    src.write_text(program)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-pthread", "-I" + CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


@pytest.mark.skipif(not shutil.which("g++"), reason="needs g++")
def test_walks_end(tmp_path):
    run(tmp_path, WALKS)


@pytest.mark.skipif(not shutil.which("g++"), reason="needs g++")
def test_nobody_is_left_at_the_vote(tmp_path):
    assert "ways to end" in run(tmp_path, PROGRAM)
