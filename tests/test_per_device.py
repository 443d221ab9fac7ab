"""CPU check of post_int4_weight_amd/csrc/per_device.hpp (plain C++, compiled here with the host compiler): what a kernel needs
set up is asked for on every device, again where it failed, and by threads that come at once. And every request for more than
64 KB of LDS goes through it: a plain flag would leave a second device without, and be written by two threads."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "post_int4_weight_amd", "csrc")

PROGRAM = r"""
#include "per_device.hpp"
#include <cstdio>
#include <thread>
#include <vector>
int main() {
    ptq::PerDevice p;
    int asked[100] = {}, bad = 0;
    auto ask = [&](int d, int status) { return p.once(d, [&] { ++asked[d]; return status; }); };
    bad += ask(3, 5) != 5 || asked[3] != 1;                    // it failed,
    bad += ask(3, 0) != 0 || asked[3] != 2;                    // is asked for again,
    bad += ask(3, 5) != 0 || asked[3] != 2;                    // and no more
    for (int d = 0; d < 64; ++d) bad += ask(d, 0) != 0 || asked[d] != (d == 3 ? 2 : 1);
    for (int d = 0; d < 64; ++d) bad += ask(d, 7) != 0 || asked[d] != (d == 3 ? 2 : 1);
    for (int i = 1; i < 4; ++i) bad += ask(64, 0) != 0 || asked[64] != i;
    ptq::PerDevice q;
    std::vector<std::thread> all;
    std::atomic<int> count[8] = {}, early{0};
    for (int t = 0; t < 16; ++t)
        all.emplace_back([&, t] {
            for (int i = 0; i < 1000; ++i) {
                const int d = (t + i) % 8;
                q.once(d, [&] { ++count[d]; return 0; });
                early += count[d] == 0;
            }
        });
    for (auto& t : all) t.join();
    for (auto& c : count) bad += c < 1 || c > 16;
    std::printf("%d\n", bad + early);
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_once_on_each_device(tmp_path):
    (tmp_path / "p.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, "-o", str(tmp_path / "p"), str(tmp_path / "p.cpp")],
                   check=True)
    assert subprocess.run([str(tmp_path / "p")], capture_output=True, text=True, check=True).stdout == "0\n"


def test_lds_is_asked_for_per_device():
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        if name != "common.hpp":
            assert "hipFuncSetAttribute" not in text, f"{name}: kernels get their LDS from allow_lds"
        assert not re.search(r"static\s+bool\s+\w+\s*=", text), f"{name}: a flag for all devices and threads"
