"""perf/operators.py: its cases hang together, and its plain form, the library's calls and the definition in 64 bits agree
on small cases of each kind."""
import importlib.util
import os
import random

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def ops():
    spec = importlib.util.spec_from_file_location("operators", os.path.join(HERE, "..", "perf", "operators.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_cases(ops):
    cases = ops.listed()
    assert 4 <= len(cases) <= 12 and len({c["name"] for c in cases}) == len(cases)
    for op in ("append", "decode", "prefill"):
        assert sum(c["op"] == op for c in cases) >= 2
    assert all(ops.work(c)["bytes"] > 0 and ops.work(c)["flops"] >= 0 for c in cases)
    drawn = [ops.draw(random.Random(i)) for i in range(50)]
    assert drawn == [ops.draw(random.Random(i)) for i in range(50)]
    assert len({str(sorted(c.items())) for c in drawn}) == 50 and all(ops.work(c)["bytes"] > 0 for c in drawn)
    assert ops.own is False


SMALL = [
    {"op": "decode", "cache": "bf16", "batch": 3, "shortest": 1, "longest": 70, "heads": 6, "kv_heads": 2, "page": 16},
    {"op": "decode", "cache": "fp8", "batch": 2, "shortest": 5, "longest": 300, "heads": 24, "kv_heads": 2, "page": 8},
    {"op": "append", "rows": "bf16", "cache": "bf16", "batch": 3, "shortest": 1, "longest": 40, "history": 5, "kv_heads": 2,
     "page": 16},
    {"op": "append", "rows": "fp8", "cache": "fp8", "batch": 4, "shortest": 1, "longest": 1, "history": 20, "kv_heads": 3,
     "page": 8},
    {"op": "append", "rows": "bf16", "cache": "fp8", "batch": 2, "shortest": 3, "longest": 90, "history": 0, "kv_heads": 2,
     "page": 32},
    {"op": "prefill", "cache": "bf16", "batch": 3, "shortest": 2, "longest": 150, "heads": 6, "kv_heads": 2, "causal": True,
     "pad_rows": 7},
    {"op": "prefill", "cache": "fp8", "batch": 2, "shortest": 9, "longest": 140, "heads": 8, "kv_heads": 2, "causal": False,
     "pad_rows": 0},
    {"op": "prefill", "cache": "fp8", "batch": 2, "shortest": 9, "longest": 140, "heads": 4, "kv_heads": 4, "causal": True,
     "pad_rows": 3},
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", SMALL, ids=lambda c: "-".join(str(c[x]) for x in ("op", "cache", "batch", "longest")))
@pytest.mark.parametrize("own", [False, True])
def test_both_forms_agree_with_the_definition(ops, monkeypatch, case, own):
    """Attention: the output's rounding, 2^-8 |o|, and for the weights and keys of the library's calls a part of the largest
    value: 2^-8 for bf16 rows; for E4M3 rows logits move by at most 2^-8 * sum |q_d k_d| / sqrt(128), below 0.05 for these
    inputs, so weights by exp(0.1) - 1.  The plain form has fp32 sums only.  Append: rows as they are, or codes that may
    differ by one step, 2^-3 of the value, where the quotient's rounding decides, and scales by 2^-22."""
    case = dict(case, lens_seed=1)
    monkeypatch.setattr(ops, "own", own)
    got, want = ops.run(ops.prepare(case, 3)), ops.exact(case, 3)
    if case["op"] != "append":
        value = 1.0 if case["cache"] == "bf16" else 1.0 + 2.0 ** -4
        largest = value * 5.5  # of some 10^5 normal numbers
        part = 2.0 ** -20 if not own else 2.0 ** -8 if case["cache"] == "bf16" else 0.11
        assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + part * largest).all()
        return
    for g, w in zip(got, want):
        err = (g.double() - w).abs()
        if g.dtype == torch.bfloat16 or case["rows"] == "fp8":
            assert (err == 0).all()
        elif g.dtype == torch.float32:
            assert (err <= 2.0 ** -22 * w).all()
        else:
            assert (err <= 2.0 ** -3 * w.abs() + 2.0 ** -9).all() and (err > 0).double().mean() < 0.01
