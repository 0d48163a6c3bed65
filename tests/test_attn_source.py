"""What the attention kernels' sources have to say, read as text: a launch that may
overlap the end of the one before it touches device memory only after its own wait."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ATTN = os.path.join(ROOT, "deterministic_fixed_order_gb300", "csrc", "attn")

# Each kernel's body and what in it reads device memory first.
BODIES = {
    "decode": ("attn_decode.cuh", "__device__ static void run("),
    "decode's join": ("attn_decode.cuh", "void join_chunks("),
    "append": ("kv_append.cu", "append_kernel("),
    "rank join": ("attn_join.cu", "join_kernel("),
}
READS = re.compile(r"\bsequence(?:_of)?<|\bbegin_walk<|\bheaders\[|\blens\[|\blses\[|\bslots\[|\bpositions\[|\bacc\[|"
                   r"\bload_q\(|\bweigh\(|\bfetch\(")


def body(file, start):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(ATTN, file)).read())
    at = text.index("{", text.index(start))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError("no end of the body")


@pytest.mark.parametrize("kernel", BODIES)
def test_kernels_wait_before_they_read(kernel):
    code = body(*BODIES[kernel])
    waits = [m.start() for m in re.finditer(r"\benter_grid\(\);", code)]
    assert len(waits) == 1, "one wait, on every path"
    before = code[:waits[0]]
    assert before.count("{") - before.count("}") == 1, "outside every branch"
    read = READS.search(code)
    assert read and read.start() > waits[0], f"{code[read.start():read.start() + 40]!r} comes before the wait"


def test_every_early_launch_is_among_them():
    kernels = set()
    for path in glob.glob(os.path.join(ATTN, "*.cu*")):
        kernels |= set(re.findall(r"launch_early\((\w+)<", open(path).read()))
    assert kernels == {"decode_kernel", "decode_join_kernel", "append_kernel", "join_kernel"}
