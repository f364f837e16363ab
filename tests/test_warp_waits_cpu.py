"""The waits of a whole warp (csrc/attn_ops.cuh) on the host: 32 threads are the lanes, polls answer each lane as
scripted, and a warp-wide instruction is a meeting that all lanes have to come to by the same kind of instruction.
Lanes whose polls differ must not part ways for good, and all must get the same answer.
"""

import os
import re
import shutil
import subprocess

import pytest

from nvfp4_kv_block_gb300 import build

HOST = r"""
#include <condition_variable>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <thread>
#include <vector>
#define __device__
#define __forceinline__ inline
struct WaitCtl { volatile int* abort; unsigned long long limit_ns; };

std::mutex mu;
std::condition_variable cv;
int come, turn, yes;
const char* kind;
int answer_all, answer_any;
unsigned long long now_ns;
thread_local int lane;
thread_local long polls;
long ready[32];  // the poll of each lane from which on it is told that the phase is there; -1: never

// All lanes come, by the same kind of instruction, or the warp would wait for good.
void meet(const char* what, bool vote, int* all, int* any) {
  std::unique_lock<std::mutex> lock(mu);
  if (come == 0) { kind = what; yes = 0; }
  if (strcmp(kind, what)) { printf("apart: %s and %s\n", kind, what); fflush(stdout); _Exit(1); }
  yes += vote;
  const int mine = turn;
  if (++come == 32) {
    answer_all = yes == 32;
    answer_any = yes > 0;
    come = 0;
    ++turn;
    cv.notify_all();
  } else {
    cv.wait(lock, [&] { return turn != mine; });
  }
  *all = answer_all;
  *any = answer_any;
}
bool vote_all(bool p) { int a, b; meet("vote", p, &a, &b); return a; }
bool vote_any(bool p) { int a, b; meet("vote", p, &a, &b); return b; }
#define __all_sync(mask, p) vote_all(p)
#define __any_sync(mask, p) vote_any(p)
#define __syncwarp() do { int a, b; meet("syncwarp", false, &a, &b); } while (0)
bool poll() { return ready[lane] >= 0 && polls++ >= ready[lane]; }
bool mbar_poll(uint32_t, uint32_t) { return poll(); }
bool mbar_try_wait(uint32_t, uint32_t) { return poll(); }
unsigned long long globaltimer_ns() { std::lock_guard<std::mutex> lock(mu); return now_ns += 10; }

WAITS

int main(int argc, char** argv) {
  for (int i = 0; i < 32; ++i) ready[i] = atol(argv[3 + i]);
  volatile int abort_flag = atoi(argv[2]);
  // (the clock goes on by 10 ns at every lane's look at it: 320 a look of the warp, every 16 or 64 polls)
  const WaitCtl w{&abort_flag, (unsigned long long)atol(argv[35])};
  int got[32];
  std::vector<std::thread> lanes;
  for (int i = 0; i < 32; ++i)
    lanes.emplace_back([&, i] {
      lane = i;
      got[i] = !strcmp(argv[1], "swait") ? swait(0, 0, w) : twait(0, 0, w);
      int a, b;
      meet("return", false, &a, &b);
    });
  for (auto& t : lanes) t.join();
  for (int i = 1; i < 32; ++i)
    if (got[i] != got[0]) { printf("lane %d got %d, lane 0 %d\n", i, got[i], got[0]); return 1; }
  printf("%d %d\n", got[0], (int)abort_flag);
  return 0;
}
"""


@pytest.fixture(scope="module")
def warp(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    with open(os.path.join(build.CSRC, "attn_ops.cuh")) as f:
        text = f.read()
    waits = [re.search(r"^__device__ __forceinline__ bool %s\(.*?^}" % name, text, re.M | re.S).group(0) for name in ("twait", "swait")]
    at = tmp_path_factory.mktemp("waits")
    (at / "w.cpp").write_text(HOST.replace("WAITS", "\n".join(waits)))
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-w", str(at / "w.cpp"), "-o", str(at / "w")], check=True)
    return lambda name, abort, ready, limit_ns: subprocess.run([str(at / "w"), name, str(abort)] + [str(x) for x in ready] + [str(limit_ns)],
                                                               capture_output=True, text=True, timeout=60)


READY = {
    "at once": [0] * 32,
    "one lane later": [0] * 31 + [1],
    "lane 0 later": [3] + [0] * 31,
    "every other lane": [i % 2 for i in range(32)],
    "each at its own poll": [7 * i % 32 for i in range(32)],
    "behind the short polls": [70 * (i % 3) for i in range(32)],
    "long apart": [0] * 16 + [1000] * 16,
}


@pytest.mark.parametrize("name", ["twait", "swait"])
@pytest.mark.parametrize("case", READY)
def test_lanes_whose_polls_differ_meet_again(warp, name, case):
    r = warp(name, 0, READY[case], 100_000)
    assert (r.returncode, r.stdout) == (0, "1 0\n"), r.stdout


@pytest.mark.parametrize("name", ["twait", "swait"])
@pytest.mark.parametrize("ready", [[-1] * 32, [0] * 31 + [-1], [-1] + [5] * 31])
def test_a_wait_that_runs_out_does_so_for_all_lanes(warp, name, ready):
    r = warp(name, 0, ready, 20_000)
    assert (r.returncode, r.stdout) == (0, "0 1\n"), r.stdout


@pytest.mark.parametrize("name", ["twait", "swait"])
def test_a_wait_ends_when_another_role_gave_up(warp, name):
    r = warp(name, 1, [-1] * 32, 20_000)
    assert (r.returncode, r.stdout) == (0, "0 1\n"), r.stdout
