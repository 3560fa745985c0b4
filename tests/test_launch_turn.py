"""The host lock over a call's launches (csrc/launch_turn.h): calls that share a
workspace take turns, others do not wait for each other."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_gemv_b200", "csrc")
PROGRAM = r"""
#include <atomic>
#include <chrono>
#include <cstdlib>
#include <thread>
#include <vector>
#include "launch_turn.h"
using qmoe::LaunchTurn;

int main()
{
    int a = 0, b = 0;
    // while one call launches, those of another workspace and of none do
    LaunchTurn first(&a);
    std::atomic<int> done{0};
    std::thread other([&] {
        { LaunchTurn t(&b); }
        { LaunchTurn t(nullptr); LaunchTurn u(nullptr); }
        done = 1;
    });
    for (int i = 0; i < 500 && !done; ++i)
        std::this_thread::sleep_for(std::chrono::milliseconds(10));
    if (!done)
        _Exit(1);
    other.join();
    // and one of the same workspace waits for it
    std::atomic<int> in{0}, out{0};
    std::thread same;
    {
        LaunchTurn mine(&b);
        same = std::thread([&] { LaunchTurn t(&b); in = out ? 1 : 2; });
        std::this_thread::sleep_for(std::chrono::milliseconds(100));
        if (in)
            _Exit(2);
        out = 1;
    }
    same.join();
    if (in != 1)
        return 3;
    // many threads, few workspaces
    std::atomic<int> inside[3] = {{0}, {0}, {0}}, bad{0};
    std::vector<std::thread> threads;
    for (int i = 0; i < 12; ++i)
        threads.emplace_back([&, i] {
            for (int k = 0; k < 5000; ++k) {
                LaunchTurn t(&inside[(i + k) % 3]);
                if (inside[(i + k) % 3]++)
                    bad = 1;
                inside[(i + k) % 3]--;
            }
        });
    for (auto &t : threads)
        t.join();
    // the process ends although a call still launches and another waits for it
    static int z = 0;
    new LaunchTurn(&z);
    std::thread([] { LaunchTurn t(&z); }).detach();
    std::this_thread::sleep_for(std::chrono::milliseconds(50));
    exit(bad ? 4 : 0);
}
"""


def test_turns(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    src = tmp_path / "turns.cpp"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I", CSRC, str(src), "-o", str(tmp_path / "turns")], check=True)
    assert subprocess.run([str(tmp_path / "turns")], timeout=60).returncode == 0
