"""The plain form of the block-table cases in perf/operators.py, run on the CPU,
against the request-by-request model that the GPU tests compare the calls with."""
import importlib.util
import os
import random

import numpy as np
import pytest
import torch

from tests.test_gpu_block_tables import extend_model, pages_of


@pytest.fixture(scope="module")
def operators():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")
    spec = importlib.util.spec_from_file_location("operators_on_cpu", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod._DEV = "cpu"
    return mod


def model(s):
    """The tables after one pass, by walking the requests."""
    bs, table, free = s["case"]["bs"], s["table"].numpy().copy(), s["free"].numpy().copy()
    lens, n_free = s["context"].numpy().copy(), int(s["num_free"])
    if s["case"]["churn"]:
        for b in np.nonzero(s["finished"].numpy())[0]:
            held = pages_of(int(lens[b]), bs)
            free[n_free:n_free + held] = table[b, :held]
            n_free += held
            lens[b] = 0
    table, lens, slots, left, status = extend_model(lens.astype(object), s["new"].numpy().astype(object), table, free, n_free,
                                                    bs, s["tokens"])
    return dict(table=table, lens=lens, slots=slots, num_free=left, free=free), status


CASES = [dict(b=66, bs=832, pages=13, prompt=49, short=0.1, churn=False),  # requests without a page after the pool has run out
         dict(b=200, bs=48, pages=9, prompt=100, short=0.1, churn=True), dict(b=5, bs=16, pages=7, prompt=90, short=0.0, churn=False),
         dict(b=1, bs=784, pages=4, prompt=1, short=0.1, churn=False)]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("seed", range(6))
def test_plain_tables_follow_the_model(operators, case, seed):
    check(operators, dict(op="tables", **case), seed)


def test_plain_tables_of_drawn_cases(operators):
    rng, done = random.Random(0), 0
    while done < 12:
        case = operators.draw(rng)
        if case["op"] == "tables" and case["b"] * case["pages"] < 100000:
            check(operators, case, done)
            done += 1


def check(operators, case, seed):
    s = operators.prepare(case, seed)
    want, _ = model(s)
    got = operators.run(s)
    for name, w in want.items():
        assert np.array_equal(got[name].numpy().reshape(np.shape(w)), w), name
