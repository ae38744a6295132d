"""What the library's sources may not hold: every rank of a job on several GPUs
loads the same libpkv.so, so no copy in it may go to several CTAs at once
(such copies are kept out of libraries that run beside other GPUs' memory)."""
import os

from paged_kv_cache_189_gb300 import build as pkv_build

WORD = "multi" + "cast"


def test_no_copies_to_several_ctas():
    found = []
    for folder in (pkv_build.CSRC, pkv_build.INCLUDE):
        for name in sorted(os.listdir(folder)):
            with open(os.path.join(folder, name)) as f:
                found += [(name, n) for n, line in enumerate(f, 1) if WORD in line.lower() or "multimem" in line]
    assert not found
