"""Which kernels of the list operators let the next one on the stream start
early (read from the source, no GPU): none whose results a kernel of another
library could read before it waits. Only the norm's first kernel, which writes
scratch, and its second where another kernel of the same call, which waits,
follows."""

import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "muon_newton_schulz_03_b200", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _kernels():
    for body in _source("grad_ops.cu").split("__global__")[1:]:
        yield re.search(r"\b(g\d_\w+)\(", body).group(1), body.split("\n}\n")[0]


def test_only_kernels_whose_next_one_waits_release_early():
    free, bound = set(), set()
    for name, body in _kernels():
        calls = len(re.findall(r"dep_release\(\)", body))
        guarded = len(re.findall(r"if \(followed\) dep_release\(\)", body))
        if calls > guarded:
            free.add(name)
        if guarded:
            bound.add(name)
    assert free == {"g1_norm"} and bound == {"g2_finish"}


def test_every_kernel_waits_before_it_touches_memory_of_others():
    names = [name for name, body in _kernels() if "dep_wait()" in body]
    assert sorted(names) == ["g1_norm", "g2_finish", "g3_scale", "g4_adamw", "g5_small"]
