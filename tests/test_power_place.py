"""Where a token's powers begin in an MXFP4 cache (CPU): against integers of any
size, over the largest caches that the calls take."""
import os
import random
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "semi_ar_draft_amd", "csrc")

PROGRAM = r"""
#include "power_place.hpp"
#include <cstdio>
int main() {
  int page, heads, head, shift, place, blocks;
  while (std::scanf("%d %d %d %d %d %d", &page, &heads, &head, &shift, &place, &blocks) == 6)
    std::printf("%lld\n", (long long)dspark::power_place(page, heads, head, shift, place, blocks));
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_places_past_32_bits(tmp_path):
    src, exe = tmp_path / "place.cpp", tmp_path / "place"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC, str(src), "-o", str(exe)],
                   check=True)
    r = random.Random(1)
    cases = [(0, 1, 0, 3, 0, 2), ((1 << 28) - 1, 1024, 1023, 3, 7, 8), (1 << 22, 1024, 0, 9, 0, 2), ((1 << 21) - 1, 1024, 1023, 10, 1023, 8)]
    for _ in range(200):
        shift, heads = r.randint(3, 10), r.randint(1, 1024)
        cases.append((r.randrange((2 ** 31 - 1) >> shift), heads, r.randrange(heads), shift, r.randrange(1 << shift), r.choice([2, 4, 8])))
    text = "\n".join(" ".join(map(str, c)) for c in cases)
    got = [int(x) for x in subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split()]
    assert got == [((p * heads + h << shift) + t) * n for p, heads, h, shift, t, n in cases]


def test_the_attention_has_no_place_of_its_own():
    text = open(os.path.join(CSRC, "attend.hip")).read()
    assert text.count("power_place(") == 2
    assert not re.search(r"a\.Hkv\s*(\*\s*power_head|<<)", text)
