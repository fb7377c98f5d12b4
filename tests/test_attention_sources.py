"""What holds for the attention kernels' source files, checked without a GPU."""
import glob
import os
import re

from gemm_epilogue_tcgen05_gb300 import build


def read(path):
    with open(path, encoding="utf-8") as f:
        return f.read()


def test_build_checks_the_registers_of_every_prefill_source():
    """Each translation unit that launches the prefill kernel holds instances of it, whose registers the build counts."""
    units = {os.path.basename(f) for f in glob.glob(os.path.join(build.ATTENTION, "*.cu")) if "launch_prefill<" in read(f)}
    assert len(units) == 3 and units == set(build.REGISTERS)


def test_attention_functions_are_reached():
    """Every device function of the attention folder has a caller there."""
    text = "\n".join(read(f) for f in glob.glob(os.path.join(build.ATTENTION, "*")) if f.endswith((".cu", ".cuh", ".h")))
    names = set(re.findall(r"__device__ __forceinline__ [\w:]+ (\w+)\(", text)) - {"operator"}
    assert len(names) > 30
    assert not [n for n in names if len(re.findall(rf"\b{n}\b", text)) < 2]


def test_products_that_round_scales_of_4_bits():
    """a times fl(1/7) rounds to the same five bits as a / 7 for every significand of a bf16 number: exactly at the two ties (231 and
    245), 1/14 of a step away from one everywhere else."""
    import numpy as np

    seventh = np.float32(1) / np.float32(7)
    ties = 0
    for a in range(128, 256):
        step = 1 if a < 7 * 32 else 2
        tie = a % 7 == 0 and (a // 7) % step != 0
        ties += tie
        got = float(np.float32(a) * seventh)
        if tie:
            assert got == a // 7
        else:
            away = abs((a - 7 * step / 2) / (7 * step) - round((a - 7 * step / 2) / (7 * step)))
            assert away >= 1 / 14 - 1e-9 and abs(got - a / 7) < 2.0 ** -18 * step
        assert round(got / step) == round(a / 7 / step)
    assert ties == 2
