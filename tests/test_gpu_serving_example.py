"""The serving example end to end: prompts, a captured decoding step replayed, and the same text as a prompt."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("args,most", [(["--batch", "4", "--prompt", "200", "--steps", "12"], 0.05),
                                       (["--batch", "1", "--prompt", "3", "--steps", "5"], 0.05),
                                       (["--batch", "3", "--prompt", "90", "--steps", "6", "--e4m3"], 0.25)])
def test_steps_continue_the_prompt(args, most):
    """The last step's logits are those of the whole text as a prompt.  Both round activations to bf16
    (2^-8) some ten times a layer, at different places, so a few percent; an e4m3 cache rounds K and V to 2^-4."""
    import decode
    assert decode.main(args) <= most
