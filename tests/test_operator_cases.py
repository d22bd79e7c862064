"""The measured cases of perf/operators.py on the CPU: their plain forms against their 64-bit references on
small drawn cases of every operator, and what they say a pass has to move."""
import importlib.util
import os
import random

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def cases():
    spec = importlib.util.spec_from_file_location("operator_cases", os.path.join(ROOT, "perf", "operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.DEV = "cpu"
    return m


def test_listed(cases):
    names = [c["name"] for c in cases.listed()]
    assert len(set(names)) == len(names) and not cases.own
    for c in cases.listed():
        w = cases.work(c)
        assert w["bytes"] > 0 and w["flops"] > 0, c


def test_work_counts(cases):
    """Bytes of three cases written out."""
    by = {c["name"]: cases.work(c)["bytes"] for c in cases.listed()}
    # x and y, the states read and written (this prompt continues sequences), weights and bias
    assert by["conv prompt 8x4096"] == 2 * 32768 * 4096 * 2 + 2 * 8 * 3 * 4096 * 2 + 4096 * 5 * 4
    # x, dt, z, y; B and C; A, D and bias; the states read and written
    assert by["scan step 256"] == 4 * 256 * 4096 * 2 + 2 * 256 * 16 * 2 + 4096 * 18 * 4 + 2 * 256 * 4096 * 16 * 4
    # x, y, the residual read and written, weights
    assert by["norm 32768x2048"] == 32768 * 2048 * (2 + 2 + 4 + 4) + 2048 * 4


def test_plain_forms(cases):
    rng, seen = random.Random(3), {}
    while len(seen) < 8 or min(seen.values()) < 2:
        c = cases.draw(rng)
        if c.get("rows", c.get("batch", c.get("tokens", 1))) * c["dim"] * c.get("dstate", 1) > 400_000:
            continue
        if seen.get(c["op"], 0) >= 3:
            continue
        want, got = cases.exact(c, 5), cases.run(cases.prepare(c, 5))
        assert set(want) == set(got), c
        for k in want:
            a, b = got[k].double(), want[k].double()
            # roundings of an output's type, or of 32 bits over a few hundred terms
            limit = {torch.float32: 1e-5, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}.get(got[k].dtype, 2.0 ** -4)
            assert a.shape == b.shape and float((a - b).norm()) <= limit * float(b.norm()) + 1e-30, (c, k)
        seen[c["op"]] = seen.get(c["op"], 0) + 1
