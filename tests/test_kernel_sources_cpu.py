"""Properties of the kernel sources that no run may show: what a fault would
need a GPU to hang or several GPUs to see is looked for in the text."""
import glob
import os
import re

from speculative_decode_hybrid_gb300 import build as B

SOURCES = sorted(glob.glob(os.path.join(B.CSRC, "*.cu")) + glob.glob(os.path.join(B.CSRC, "*.cuh")))


def code(path):
    """The file without comments, adjacent string literals joined."""
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.sub(r'"\s*\n\s*"', "", text)


def test_no_load_is_multicast():
    """The library is one file for programs on one GPU and on several: a bulk
    load that a cluster shares has no place in it."""
    assert SOURCES
    for path in SOURCES:
        for copy in re.findall(r'"[^"]*cp\.async\.bulk[^"]*"', code(path)):
            assert "multicast" not in copy, (os.path.basename(path), copy)


def test_attention_takes_tensor_memory_after_the_grid_wait():
    """A block that holds all of an SM's columns while it waits for the kernel
    before would hang with one that allocates after letting it start."""
    text = code(os.path.join(B.CSRC, "attn_tc.cu"))
    assert text.count("tmem_alloc") == 1 and 0 < text.index("pdl_wait()") < text.index("tmem_alloc")


def test_the_number_of_sms_is_asked_for():
    """152 stands only where the device does not answer."""
    for path in SOURCES:
        for line in code(path).splitlines():
            if re.search(r"\b(152|304)\b", line):
                assert re.search(r"sms (> 0 \?|<= 0 \? 152)", line), (os.path.basename(path), line.strip())
