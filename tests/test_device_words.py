"""The device words that a context's launches share (CPU): every user has its
own, also against what the chained draft's merge clears."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "semi_ar_draft_amd", "csrc")

PROGRAM = r"""
#include "device_words.hpp"
#include <cstdio>
using namespace dspark;
int main() {
  std::printf("%zu %zu %zu %zu %zu %d %d\n", offsetof(DeviceWords, err), offsetof(DeviceWords, bar),
              offsetof(DeviceWords, pages_done), offsetof(DeviceWords, chain), sizeof(DeviceWords), kChainFirst, kChainCounters);
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_no_word_has_two_users(tmp_path):
    src, exe = tmp_path / "words.cpp", tmp_path / "words"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    err, bar, pages, chain, size, first, counters = map(int, out.split())
    cleared = {chain // 4} | set(range(chain // 4 + first, chain // 4 + first + counters))
    singles = {err // 4, bar // 4, pages // 4}
    assert len(singles) == 3 and not singles & cleared
    assert max(cleared | singles) < size // 4
    assert counters >= 2 * 32                                     # two groups of 32 positions


def test_the_kernels_clear_what_the_block_holds():
    """The merges and the ticket code index the counters by the block's own constants."""
    for name in ("sweep.hip", "confidence.hip"):
        text = open(os.path.join(CSRC, name)).read()
        assert "threadIdx.x <= kChainCounters" in text and "kChainFirst - 1 + threadIdx.x" in text, name
