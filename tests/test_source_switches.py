"""Every macro that the sources test is defined somewhere in the tree, or by the compiler (CPU)."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "linear_recurrent_sequence_causal_gb300")
COMPILERS = {"__cplusplus", "__CUDACC__", "__CUDA_ARCH__", "__GNUC__"}


def test_no_switch_without_a_hand_on_it():
    files = [*glob.glob(os.path.join(PKG, "csrc", "*")), *glob.glob(os.path.join(ROOT, "include", "*.h")), os.path.join(PKG, "build.py")]
    text = {f: open(f).read() for f in files}
    every = "\n".join(text.values())
    for f, src in text.items():
        for line in re.findall(r"^\s*#\s*(?:if|ifdef|ifndef|elif)\b(.*)$", src, re.M):
            for name in re.findall(r"[A-Za-z_]\w*", line):
                if name != "defined" and name not in COMPILERS:
                    assert re.search(rf"#\s*define\s+{name}\b|-D{name}\b", every), f"{os.path.basename(f)} tests {name}, which nothing defines"
