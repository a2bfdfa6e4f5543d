"""The plain forms of perf/operators.py on the CPU: a call leaves its inputs as
they were (only what the operator updates by its definition changes), so every
call on one state of an operator without such an update gives the same answer;
and the answer is the 64-bit definition's.

Tolerance of the fp32 forms against 64 bits: sums of at most 64 tokens whose
terms are each off by a few roundings of 2^-24, relative to the largest value:
64 * 4 * 2^-24 = 2^-16.
"""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def operators(monkeypatch):
    spec = importlib.util.spec_from_file_location("measured_operators", os.path.join(ROOT, "perf", "operators.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    monkeypatch.setattr(module, "DEV", "cpu")
    return module


def diag(**kw):
    return dict(dict(op="diag", B=2, T=10, C=24, dtype="f32", mix=False, train=True), **kw)


REPEATED = [
    diag(), diag(mix=True), diag(dtype="bf16"), diag(dtype="bf16", mix=True), diag(train=False), diag(B=1, T=1),
    diag(B=3, T=64, mix=True),
    dict(op="attn", B=2, T=1, Hq=4, Hkv=2, D=64, page=16, past=40, window=0),
    dict(op="attn", B=2, T=9, Hq=4, Hkv=2, D=64, page=16, past=40, window=12),
]
UPDATING = [   # and what the operator updates in place
    (dict(op="step", B=3, H=4, d=64, delta=False, slots=False), {"S"}),
    (dict(op="step", B=3, H=4, d=64, delta=True, slots=True), {"S"}),
    (dict(op="append", B=3, T=20, Hq=4, Hkv=2, D=64, page=16, past=21, rot=32, inter=True), {"kc", "vc", "ks", "vs"}),
]


def bits(t):
    return t.contiguous().view(torch.uint8)


def held(state):
    return {k: t.clone() for k, t in state.items() if isinstance(t, torch.Tensor)}


@pytest.mark.parametrize("case", REPEATED, ids=[str(i) for i in range(len(REPEATED))])
def test_plain_calls_repeat_and_leave_their_inputs(operators, case):
    state = operators.prepare(case, 5)
    before = held(state)
    first = [t.clone() for t in operators.run(state)]
    second = operators.run(state)
    for a, b in zip(first, second):
        assert torch.equal(bits(a), bits(b))
    for name, t in before.items():
        assert torch.equal(bits(t), bits(state[name])), name


@pytest.mark.parametrize("case,updated", UPDATING, ids=[str(i) for i in range(len(UPDATING))])
def test_plain_calls_change_only_what_they_update(operators, case, updated):
    state = operators.prepare(case, 5)
    before = held(state)
    operators.run(state)
    for name, t in before.items():
        assert torch.equal(bits(t), bits(state[name])) == (name not in updated), name


@pytest.mark.parametrize("case", [c for c in REPEATED if c.get("dtype") == "f32"],
                         ids=lambda c: f"{c['B']}x{c['T']}-{'mix' if c['mix'] else 'plain'}-{c['train']}")
def test_later_fp32_calls_are_the_definition(operators, case):
    state = operators.prepare(case, 6)
    want = operators.exact(case, 6)
    for _ in range(3):
        got = operators.run(state)
        assert len(got) == len(want)
        for g, w in zip(got, want):
            assert (g.double() - w).abs().max() <= 2.0 ** -16 * w.abs().max()
