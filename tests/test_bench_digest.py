"""The digest that ties bench.py's recorded DRAM traffic to the kernel it was
taken on covers what the fixed-batch attention kernels are built from, and
nothing else."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)


def _digest(files):
    import bench

    return bench.kernel_sources_digest(lambda n: list(files) if n is None else files[n])


FILES = {"attn_fwd.cu": b'#include <cuda.h>\n#include "a.h"\n', "attn_pp.cu": b'  # include "b.cuh"\n', "a.h": b'#include "c.h"\n',
         "b.cuh": b'#include "zattn.h"\n', "c.h": b'#include "a.h"\n', "serving.h": b'#include "c.h"\n', "decode.cu": b'#include "serving.h"\n'}


def test_digest_follows_the_includes():
    d = _digest(FILES)
    for n in ("attn_fwd.cu", "attn_pp.cu", "a.h", "b.cuh", "c.h"):
        assert _digest({**FILES, n: FILES[n] + b"// changed"}) != d, n
    for n in ("serving.h", "decode.cu"):
        assert _digest({**FILES, n: FILES[n] + b"// changed"}) == d, n


def test_sources_of_other_operators_are_not_in_it():
    import bench

    csrc = os.path.join(ROOT, "bf16_causal_prefill_02_b200", "csrc")
    files = {}
    for n in os.listdir(csrc):
        if n.endswith((".cu", ".cuh", ".h")):
            with open(os.path.join(csrc, n), "rb") as f:
                files[n] = f.read()
    d = _digest(files)
    assert d == bench.kernel_sources_digest()
    of_it = {n for n in files if _digest({**files, n: files[n] + b"//"}) != d}
    assert of_it == {"attn_fwd.cu", "attn_pp.cu", "attn_math.cuh", "schedule.h", "sm100_ptx.cuh", "zq_internal.h"}
