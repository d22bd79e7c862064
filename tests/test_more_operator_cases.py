"""The measured cases of perf/more_operators.py on the CPU: their plain forms against their 64-bit references on
small drawn cases of every operator, and what they say a pass has to move."""
import importlib.util
import os
import random

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def cases():
    spec = importlib.util.spec_from_file_location("more_operator_cases", os.path.join(ROOT, "perf", "more_operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.DEV = "cpu"
    return m


def test_work_counts(cases):
    """Bytes of five cases written out."""
    names = [c["name"] for c in cases.listed()]
    assert len(set(names)) == len(names) == 12 and not cases.own
    by = {c["name"]: cases.work(c)["bytes"] for c in cases.listed()}
    # x, gate, i, y; weight; the last states written
    assert by["gated prompt 8x4096"] == 4 * 32768 * 4096 * 2 + 4096 * 4 + 8 * 4096 * 4
    # x, gate, z, y; weight; the states read and written
    assert by["gated step 256"] == 4 * 256 * 4096 * 2 + 4096 * 4 + 2 * 256 * 4096 * 4
    # x, gate, i, dy read, dx, dgate, di written; weight and its gradient
    assert by["gated backward 8x2048"] == 7 * 16384 * 4096 * 2 + 2 * 4096 * 4
    # x, z, y; weight, bias
    assert by["group norm 32768x2048"] == 3 * 32768 * 2048 * 2 + 2 * 2048 * 4
    # states read, bytes and scales written; bytes and scales read again by the load are the cache's own
    assert by["cache int8 64"] == 64 * 262144 * (4 + 1 + 4) + 64 * 4096 * 4


def test_plain_forms(cases):
    rng, seen = random.Random(3), {}
    while len(seen) < 7 or min(seen.values()) < 3:
        c = cases.draw(rng)
        n = c.get("rows", c.get("batch", c.get("tokens", c.get("count")))) * \
            c.get("dim", c.get("values", c.get("groups", 1) * c.get("size", 1)))
        if n > 200_000 or seen.get(c["op"], 0) >= 4:
            continue
        want, got = cases.exact(c, 5), cases.run(cases.prepare(c, 5))
        if torch.is_tensor(want):
            want, got = dict(y=want), dict(y=got)
        assert set(want) == set(got), c
        for k in want:
            a, b = got[k].double(), want[k].double()
            # roundings of an output's type, or of 32 bits over a few hundred terms
            limit = {torch.float32: 1e-5, torch.bfloat16: 2.0 ** -8}[got[k].dtype]
            assert a.shape == b.shape and float((a - b).norm()) <= limit * float(b.norm()) + 1e-30, (c, k)
        seen[c["op"]] = seen.get(c["op"], 0) + 1
