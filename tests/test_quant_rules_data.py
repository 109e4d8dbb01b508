"""The rules by which the 8-bit operators and the expert layer choose their
kernels, against the times of every variant that tests/data/
quant_rules_gfx950.json holds: how much longer the choice takes than the
fastest variant, on average and at worst.

The limits are what the rules reach on these times (in the test's own
arithmetic), rounded up: a rule or a table that gets worse shows here.  (The
expert layer's worst are experts of 1024, 512, where the wide form's three
further launches weigh most.)"""
import json
import os

import pytest

import block_wise_int4_matmulnbits_amd as mnb
from tests import quant_routes

DATA = os.path.join(os.path.dirname(os.path.abspath(__file__)), "data", "quant_rules_gfx950.json")
LAUNCH = 2.0   # us that one more launch costs a call besides its kernel's time


@pytest.fixture(scope="module")
def routes(tmp_path_factory):
    return quant_routes.Routes(tmp_path_factory.mktemp("routes"))


def _excess(rule, choices):
    """(mean, worst) of the chosen variant's time over the fastest one's."""
    with open(DATA) as f:
        entries = json.load(f)[rule]
    shapes = [tuple(k) for k, _ in entries]
    ratios = []
    for (_, times), choice in zip(entries, choices(shapes)):
        us = {v: sum(t) + LAUNCH * (len(t) - 1) if isinstance(t, list) else t for v, t in times.items()}
        ratios.append(us[choice] / min(us.values()))
    return sum(ratios) / len(ratios), max(ratios)


RULES = {
    "int8_tile": (lambda r, s: [t for t, _, _, _ in r.int8([(mnb.MNB_I8,) + k for k in s])], 1.002, 1.04),
    "int8_rows_waves": (lambda r, s: ["8" if w <= 8 else "16" for _, w, _, _ in r.int8([(mnb.MNB_I8,) + k for k in s])],
                        1.006, 1.07),
    "int8_fuse": (lambda r, s: ["one" if f else "two" for _, _, _, f in r.int8([(mnb.MNB_F16,) + k for k in s])],
                  1.005, 1.10),
    "quantize": (lambda r, s: r.quantize(s), 1.008, 1.21),
    "moe_kernels": (lambda r, s: [c for c, _ in r.moe_choice(s)], 1.034, 1.32),
    "moe_down_quads": (lambda r, s: [q for _, q in r.moe_choice(s)], 1.001, 1.01),
}


@pytest.mark.parametrize("rule", sorted(RULES))
def test_choice_is_near_the_fastest(rule, routes):
    choices, mean, worst = RULES[rule]
    got = _excess(rule, lambda shapes: choices(routes, shapes))
    assert got[0] <= mean and got[1] <= worst, got
