"""The bounded waits of the tensor-core kernels, compiled for the host with a
stand-in barrier (CPU): no copy is left under way by a wait that was given up."""
import os
import re
import shutil
import subprocess

import pytest

from speculative_decoding_tree_gb300 import _build

HOST = r"""
#include <cstdint>
#include <cstdio>
static uint64_t now = 0, ready = 0;              // a clock that each look advances; when the copy has landed
static uint64_t globaltimer_ns() { return now += 10; }
static bool mbar_try_wait(uint32_t, uint32_t) { return (now += 10) >= ready; }
%s
int main() {
  // copy lands at 500 of a limit of 1000: nobody gives up; another role has given up; the copy never lands
  const uint64_t never = 1ull << 60;
  struct { uint64_t at; int flag; } cases[] = {{500, 0}, {500, 1}, {1500, 0}, {never, 0}, {never, 1}};
  for (auto& c : cases) {
    now = 0;
    ready = c.at;
    volatile int flag = c.flag;
    const bool ok = mbar_wait_landed(0, 0, &flag, 1000);
    std::printf("%%d %%d %%d %%d\n", (int)ok, (int)flag, (int)(now >= ready), (int)(now <= 2300));
  }
  now = 0;
  wait_ns(1000);
  std::printf("%%d\n", (int)(now >= 1000 && now <= 1100));
}
"""


def function(name, text):
    """The source of a function of one brace level, without its qualifiers."""
    at = re.search(r"__device__ __forceinline__ (\w+ %s\()" % name, text)
    assert at, name
    body = text[at.start(1):]
    return "static " + body[:body.index("\n}\n") + 3]


def test_a_copy_lands_before_its_cta_leaves(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    text = open(os.path.join(_build.CSRC, "tc_ptx.cuh")).read()
    src = tmp_path / "waits.cpp"
    src.write_text(HOST % "\n".join(function(n, text) for n in ("mbar_wait", "mbar_wait_landed", "wait_ns")))
    subprocess.run([gxx, "-std=c++17", str(src), "-o", str(tmp_path / "waits")], check=True)
    out = subprocess.run([str(tmp_path / "waits")], capture_output=True, text=True, check=True).stdout.split("\n")
    # returned, abort flag, landed by then, within two limits
    assert out[:5] == ["1 0 1 1", "0 1 1 1", "0 1 1 1", "0 1 0 1", "0 1 0 1"] and out[5] == "1"


@pytest.mark.parametrize("name", ["tv_prompt_tc.cu", "tv_prompt_tc2.cu", "tv_attn_tc2.cu", "tv_attn_tcp.cu"])
def test_producers_wait_for_the_copies_of_tails(name):
    """A V tile whose rows past the end become zeros is waited for before its step counts as issued."""
    text = open(os.path.join(_build.CSRC, name)).read()
    assert text.count("mbar_wait_landed(TAIL") == 1 and "mbar_wait(TAIL" not in text
