"""The 4-bit cache's kernels are launched while the stream's last kernel still runs, which may be writing what they
read: none of their loads may take the read-only path, which the compiler may move before the wait for that kernel."""
import glob
import os
import re

from gqa_decoder_forward_gb300 import build


def test_no_load_of_the_4_bit_kernels_is_free_to_move_before_the_wait():
    files = sorted(glob.glob(os.path.join(build.CSRC, "kv4*")))
    assert len(files) >= 4
    found = [f"{os.path.basename(f)}: {m}" for f in files
             for m in re.findall(r"__ld[a-z]+\(|__restrict__|asm\(\"ld\.|ld\.global\.nc\.[a-z0-9.]+ %", open(f).read())]
    assert not found, found
