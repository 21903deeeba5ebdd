"""The serving example over a 4-bit cache, and with several pages taken while a captured step is replayed."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("args,most", [(["--batch", "3", "--prompt", "90", "--steps", "6", "--e2m1"], 0.25),
                                       (["--batch", "2", "--prompt", "1", "--steps", "40"], 0.05),
                                       (["--batch", "5", "--prompt", "150", "--steps", "20", "--e2m1"], 0.25)])
def test_steps_continue_the_prompt(args, most):
    """As of the 16-bit cache; over 4 bits an activation that rounds to another 16-bit value can round to another code, a
    quarter of a value away."""
    import decode
    assert decode.main(args) <= most
