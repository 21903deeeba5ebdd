"""The serving example's prompts come from its own seed, and its steps continue any of them."""
import functools
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("cache", [[], ["--e4m3"], ["--e2m1"]])
def test_a_run_repeats_itself(cache):
    """Whatever the program drew before: the same prompts, steps and logits."""
    import decode
    args, got = ["--batch", "2", "--prompt", "30", "--steps", "4", *cache], []
    for seed in (1, 2):
        torch.manual_seed(seed)
        got.append(decode.main(args))
    assert got[0] == got[1] and decode.main([*args, "--seed", "5"]) != got[0]


@pytest.mark.parametrize("cache", [[], ["--e4m3"]])
def test_steps_continue_any_prompt(monkeypatch, cache):
    """With every expert chosen no rounding can choose another.  Activations are then rounded to bf16 some ten times in each of
    two layers on either way, by 2^-9 of their size on average: together at most 20 times 2^-9, if no two cancel."""
    import decode
    monkeypatch.setattr(decode, "Decoder", functools.partial(decode.Decoder, experts=8, topk=8))
    for seed in range(12):
        assert decode.main(["--batch", "2", "--prompt", "40", "--steps", "8", "--seed", str(seed), *cache]) <= 20 * 2.0 ** -9
