"""perf/more_operators.py: its cases hang together, and its plain form, the library's calls and the definition in 64 bits agree
on small cases of each kind."""
import importlib.util
import os
import random

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def ops():
    spec = importlib.util.spec_from_file_location("more_operators", os.path.join(HERE, "..", "perf", "more_operators.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_cases(ops):
    cases = ops.listed()
    assert 4 <= len(cases) <= 12 and len({c["name"] for c in cases}) == len(cases)
    for op in ("append", "decode", "prefill", "read", "step"):
        assert sum(c["op"] == op for c in cases) >= (1 if op == "step" else 2)
    assert all(ops.work(c)["bytes"] > 0 and ops.work(c)["flops"] >= 0 for c in cases)
    drawn = [ops.draw(random.Random(i)) for i in range(50)]
    assert drawn == [ops.draw(random.Random(i)) for i in range(50)]
    assert len({str(sorted(c.items())) for c in drawn}) == 50 and all(ops.work(c)["bytes"] > 0 for c in drawn)
    assert ops.own is False


SMALL = [
    {"op": "decode", "cache": "int4", "batch": 3, "shortest": 1, "longest": 300, "heads": 6, "kv_heads": 2, "page": 16,
     "window": 0, "sinks": 0},
    {"op": "decode", "cache": "int4", "batch": 4, "shortest": 9, "longest": 290, "heads": 24, "kv_heads": 2, "page": 5,
     "window": 33, "sinks": 3},
    {"op": "decode", "cache": "bf16", "batch": 2, "shortest": 40, "longest": 200, "heads": 4, "kv_heads": 4, "page": 32,
     "window": 50, "sinks": 0},
    {"op": "step", "cache": "int4", "batch": 5, "shortest": 1, "longest": 150, "heads": 8, "kv_heads": 2, "page": 8,
     "window": 0, "sinks": 0},
    {"op": "append", "cache": "int4", "batch": 3, "shortest": 1, "longest": 90, "history": 7, "kv_heads": 3, "page": 16},
    {"op": "read", "cache": "int4", "batch": 3, "shortest": 1, "longest": 90, "kv_heads": 2, "page": 16},
    {"op": "read", "cache": "fp8", "batch": 2, "shortest": 3, "longest": 60, "kv_heads": 5, "page": 8},
    {"op": "read", "cache": "bf16", "batch": 2, "shortest": 3, "longest": 60, "kv_heads": 1, "page": 1},
    {"op": "prefill", "cache": "bf16", "batch": 3, "shortest": 2, "longest": 150, "heads": 6, "kv_heads": 2, "window": 40,
     "sinks": 2, "history": 0, "pad_rows": 7},
    {"op": "prefill", "cache": "fp8", "batch": 2, "shortest": 9, "longest": 140, "heads": 8, "kv_heads": 2, "window": 30,
     "sinks": 0, "history": 100, "pad_rows": 3},
    {"op": "prefill", "cache": "bf16", "batch": 2, "shortest": 1, "longest": 70, "heads": 4, "kv_heads": 1, "window": 0,
     "sinks": 0, "history": 200, "pad_rows": 0},
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", SMALL, ids=lambda c: "-".join(str(c[x]) for x in ("op", "cache", "batch", "longest")))
@pytest.mark.parametrize("own", [False, True])
def test_both_forms_agree_with_the_definition(ops, monkeypatch, case, own):
    """Attention: the output's rounding, 2^-8 |o|, and for the weights and keys of the library's calls a part of the largest
    value: 2^-8 for weights in bf16; over 4 bits 2^-10 for the two roundings to fp16 and 2 * 300 keys * 2^-24 * 23 scales of a
    seventh of a value, 2^-9 together; for E4M3 rows logits move by at most 2^-8 * sum |q_d k_d| / sqrt(128), below 0.05 for
    these inputs, so weights by exp(0.1) - 1.  The plain form has fp32 sums only.  What 4 bits hold, and rows that come back
    from them or from bf16, are exact; E4M3 entries come back rounded once, 2^-8 of the value."""
    case = {"lens_seed": 1, "history": 0} | case
    monkeypatch.setattr(ops, "own", own)
    got, want = ops.run(ops.prepare(case, 3)), ops.exact(case, 3)
    if case["op"] in ("append", "read"):
        for g, w in zip(got, want, strict=True):
            assert ((g.double() - w).abs() <= (2.0 ** -8 * w.abs() if case["cache"] == "fp8" else 0.0)).all()
        return
    if case["op"] == "step":
        assert all(torch.equal(g.double(), w) for g, w in zip(got[1:], want[1:], strict=True))
        got, want = got[0], want[0]
    value = 1.0 if case["cache"] == "bf16" else 1.0 + 2.0 ** -4
    largest = value * 5.5  # of some 10^5 normal numbers
    part = 2.0 ** -20 if not own else {"bf16": 2.0 ** -8, "int4": 2.0 ** -9, "fp8": 0.11}[case["cache"]]
    assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + part * largest).all()
