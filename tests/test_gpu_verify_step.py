"""The cache operators and the INT4 products together, as a decoding loop uses
them: speculative decoding with draft trees says what one token at a time says."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "verify_step.py")


def test_speculative_decoding_agrees_with_stepwise():
    spec = importlib.util.spec_from_file_location("verify_step", EXAMPLE)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    gen = torch.Generator().manual_seed(5)
    prompts = [torch.randint(0, ex.VOCAB, (n,), generator=gen).cuda() for n in (37, 90)]
    model = ex.Model()
    steps = 24
    want = ex.stepwise(model, prompts, steps)
    said, verifies = ex.speculative(model, prompts, steps, want)
    assert said == want
    assert verifies < steps - 1  # trees were accepted
    assert len(set(want[0] + want[1])) > steps  # and the model does listen to its context
    # an 8-bit cache: the whole loop runs, no index leaves its buffers, and both ways begin alike
    want = ex.stepwise(model, prompts, 4, True)
    assert [s[0] for s in ex.speculative(model, prompts, 4, want, True)[0]] == [s[0] for s in want]
