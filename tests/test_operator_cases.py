"""The calls that perf/more_operators.py makes, for cases it may draw (CPU only: the calls
are recorded in place of being made)."""
import importlib.util
import os
import random

import torch

from combine_ep_layout_10_amd import ops

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "more_operators.py")


def test_sequences_go_with_the_loss(monkeypatch):
    """A gradient without the loss's counts is called without seq_off, which ep_route_backward refuses then."""
    spec = importlib.util.spec_from_file_location("more_operators", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.own = True
    made = []
    monkeypatch.setattr(ops, "route_backward", lambda *a, **kw: made.append(kw))
    rng, seen = random.Random(5), set()
    for case in m.listed() + [m.draw(rng) for _ in range(600)]:
        if case["op"] != "backward":
            continue
        state = dict(case=case, router=None, logits=None, idx=None, grad_w=torch.ones(1),
                     seq_off=torch.zeros(case["sequences"] + 1) if case["sequences"] > 1 else None)
        if case["loss"]:
            state.update(counts=torch.ones(1), coef=torch.ones(1), grad_loss=torch.ones(()))
        m.run(state)
        given = made.pop()
        assert (given["counts"] is not None) == case["loss"]
        assert (given["seq_off"] is not None) == (case["loss"] and case["sequences"] > 1)
        seen.add((case["loss"], case["sequences"] > 1))
    assert seen == {(a, b) for a in (True, False) for b in (True, False)}
