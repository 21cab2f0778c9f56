"""Drawn cases of sampling and sequence extension: the binding's calls against the plain forms of
perf/more_operators.py, both on one prepared state, whole numbers for whole numbers.

    python -m tests.drawn_cases --seed 1 --count 1000

A token that differs is looked at in 64 bits with the bound that the header gives (either of two
neighbours is right where the random point or top-p's share lies on their border); anything else
that differs ends the run.
"""
from __future__ import annotations

import argparse
import random

import torch

from perf import more_operators as P
from tests import loop_ref as R


def _outputs(state, own):
    P.own = own
    try:
        out = P.run(state)
    finally:
        P.own = False
    return [t.clone() for t in (out.values() if isinstance(out, dict) else out)]


def _sample(c, s):
    """The number of rows at a border where the forms take different neighbours."""
    (want, _), (tok, lp) = _outputs(s, False), _outputs(s, True)
    rows = (want != tok).nonzero()[:, 0]

    def of(t, i):
        return None if t is None else t[i]

    # some rows in 64 bits whatever the plain form says, for their log probabilities
    rows = torch.cat([rows, torch.arange(min(c["B"], 2), device=rows.device)])
    R.check_draws(s["x"][rows], tok[rows], lp[rows], s["bits"][rows], of(s["temp"], rows),
                  of(s["k"], rows), of(s["p"], rows), of(s["m"], rows))
    return int((want != tok).sum())


def _extend(c, s):
    written = [s[name] for name in ("out_lens", "out_count", "qsl", "slots", "pos")]
    tables, results = s["bt"].clone(), []
    for own in (False, True):
        s["bt"].copy_(tables)
        for t in written:
            t.fill_(-7)
        results.append(_outputs(s, own))
    for x, y in zip(*results):
        assert torch.equal(x, y), c
    return 0


def compare(seed, count, say=None):
    """`count` drawn cases of the two operators; returns (cases of each, rows, rows at borders)."""
    from paged_kv_attention_18_gb300 import binding
    r = random.Random(seed)
    cases, rows, borders = {"sample": 0, "extend": 0}, 0, 0
    while sum(cases.values()) < count:
        c = P.draw(r)
        if c["op"] not in cases:
            continue
        s = P.prepare(c, r.randrange(1 << 30))
        borders += (_sample if c["op"] == "sample" else _extend)(c, s)
        torch.cuda.synchronize()
        assert binding.device_error() == 0, c
        cases[c["op"]] += 1
        rows += c["B"]
        if say and sum(cases.values()) % 500 == 0:
            say(cases, rows, borders)
    return cases, rows, borders


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    a.add_argument("--seed", type=int, default=1)
    a.add_argument("--count", type=int, default=1000)
    a = a.parse_args()

    def say(cases, rows, borders):
        print(f"{cases['sample']} cases of sampling, {cases['extend']} of extension, {rows} rows: "
              f"{borders} at a border of two tokens, all others the same", flush=True)

    say(*compare(a.seed, a.count, say))
