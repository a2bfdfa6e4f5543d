"""The plain forms of perf/more_operators.py on the CPU: a call leaves its inputs as
they were (only what the operator updates by its definition changes), every call
on one state of an operator without such an update gives the same answer, and the
answer is the 64-bit definition's; the drawn cases are those of the stated ranges.

Tolerance of the fp32 forms against 64 bits: sums of at most 64 tokens, 64 states or
64 channels whose terms are each off by a few roundings of 2^-24, relative to the
largest value: 64 * 8 * 2^-24 = 2^-15.
"""
import importlib.util
import os
import random

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def operators(monkeypatch):
    spec = importlib.util.spec_from_file_location("more_measured_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    monkeypatch.setattr(module, "DEV", "cpu")
    return module


def conv(**kw):
    return dict(dict(op="conv", kind="train", B=3, T=11, C=24, K=4, dtype="f32", act=True, ragged=False), **kw)


def scan(**kw):
    return dict(dict(op="scan", kind="train", B=3, T=11, C=32, N=8, G=1, dtype="f32", gate=True, ragged=False), **kw)


CASES = [conv(), conv(ragged=True, K=2), conv(kind="piece", act=False, C=19), conv(dtype="bf16", T=40), conv(kind="piece", T=1, B=1),
         scan(), scan(ragged=True, G=2), scan(kind="piece", gate=False, C=19), scan(dtype="bf16", N=16, T=40), scan(kind="piece", T=1, B=1)]
TOKENS = [conv(kind="token", T=1), conv(kind="token", T=3, ragged=True), scan(kind="token", T=1), scan(kind="token", T=3, ragged=True)]


def bits(t):
    return t.contiguous().view(torch.uint8)


def held(state):
    flat = {k: t for k, t in state.items() if isinstance(t, torch.Tensor)} | state["out"]
    return {k: t.clone() for k, t in flat.items()}


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_plain_calls_repeat_and_leave_their_inputs(operators, case):
    state = operators.prepare(case, 5)
    before = held(state)
    first = [t.clone() for t in operators.run(state)]
    for a, b in zip(first, operators.run(state)):
        assert torch.equal(bits(a), bits(b))
    for name, t in held(state).items():
        assert torch.equal(bits(t), bits(before[name])), name


@pytest.mark.parametrize("case", TOKENS, ids=[str(i) for i in range(len(TOKENS))])
def test_plain_tokens_change_their_states_alone(operators, case):
    state = operators.prepare(case, 5)
    before = held(state)
    operators.run(state)
    for name, t in held(state).items():
        assert torch.equal(bits(t), bits(before[name])) == (name != "S"), name


@pytest.mark.parametrize("case", [c for c in CASES + TOKENS if c["dtype"] == "f32"], ids=lambda c: f"{c['op']}-{c['kind']}-{c['T']}-{c['ragged']}")
def test_plain_calls_are_the_definition(operators, case):
    got, want = operators.run(operators.prepare(case, 6)), operators.exact(case, 6)
    assert len(got) == len(want)
    for g, w in zip(got, want):
        assert g.shape == w.shape and (g.double() - w).abs().max() <= 2.0 ** -15 * w.abs().max()


def test_cases(operators):
    listed = operators.listed()
    assert len({c["name"] for c in listed}) == len(listed) and {c["op"] for c in listed} == {"conv", "scan"}
    size = lambda c: c["B"] * c["T"] * c["C"] * c.get("N", 1)  # noqa: E731
    most = {op: max(size(c) for c in listed if c["op"] == op) for op in ("conv", "scan")}
    rng = random.Random(7)
    for _ in range(200):
        c = operators.draw(rng)
        assert 1 <= c["C"] <= 4096 and c["T"] >= 1 and c["B"] >= 1 and size(c) <= most[c["op"]]
        assert c["op"] == "conv" or c["C"] % c["G"] == 0 and (c["G"] == 1 or c["C"] // c["G"] % 8 == 0)
