"""The rules by which the cache, attention and adapter calls choose their kernels
and layouts, against the times of every variant that tests/data/
kv_rules_gfx950.json holds: how much longer the choice takes than the fastest
variant, on average and at worst.

The limits are what the rules reach on these times, rounded up: a rule that gets
worse shows here.  (attention_many_rows goes by the batch's rows and heads alone,
as lengths are on the device: where some hundred rows see a few hundred keys, the
kernels of few rows would take half as long, and over 32768 keys the tiles.)"""
import json
import os

import pytest

from tests import kv_routes

DATA = os.path.join(os.path.dirname(os.path.abspath(__file__)), "data", "kv_rules_gfx950.json")

LIMITS = {      # mean, worst
    "append_threads": (1.007, 1.30),
    "attention_many_rows": (1.12, 2.40),
    "attention_cut": (1.02, 1.25),
    "attention_shares": (1.04, 1.26),
    "lora_up": (1.025, 1.31),
    "lora_up_few": (1.002, 1.04),
    "lora_down": (1.02, 1.13),
    "lora_splits": (1.015, 1.08),
}


@pytest.fixture(scope="module")
def routes(tmp_path_factory):
    return kv_routes.Routes(tmp_path_factory.mktemp("routes"))


@pytest.fixture(scope="module")
def data():
    with open(DATA) as f:
        return json.load(f)


@pytest.mark.parametrize("rule", sorted(LIMITS))
def test_choice_is_near_the_fastest(rule, routes, data):
    shapes, times = zip(*data[rule])
    choices = getattr(routes, "lora_up" if rule == "lora_up_few" else rule)(shapes)
    ratios = [us[c] / min(us.values()) for us, c in zip(times, choices)]
    mean, worst = sum(ratios) / len(ratios), max(ratios)
    assert mean <= LIMITS[rule][0] and worst <= LIMITS[rule][1], (mean, worst)


def test_other_choices_are_worse(data):
    """No one variant everywhere does as well as a rule that chooses."""
    for rule in ("append_threads", "attention_many_rows", "attention_cut", "lora_up", "lora_up_few", "lora_down"):
        for v in data[rule][0][1]:
            mean = sum(us[v] / min(us.values()) for _, us in data[rule]) / len(data[rule])
            assert mean > LIMITS[rule][0], (rule, v, mean)
