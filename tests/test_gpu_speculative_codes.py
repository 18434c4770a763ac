"""The operators together over an 8-bit cache (examples/speculative_decode.py --codes): drafts that are right are taken."""
import os
import sys

import pytest
import torch

from mixture_experts_ffn_moe_gb300 import build
from test_gpu_speculative_decode import follow

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


@pytest.mark.parametrize("hit", [0.0, 0.7, 1.0])
def test_drafted_decoding_over_codes_takes_the_models_best_tokens(hit):
    import speculative_decode as sd
    plain, steps = sd.generate(sd.Model(2, codes=True), 7, 30)
    assert steps == 30
    drafted, steps = sd.generate(sd.Model(2, codes=True), 7, 30, known=plain, hit=hit, seed=3)
    if hit == 1.0:
        # five tokens a step as long as what is decoded is what the drafts know; from the first token on that rounding decided
        # otherwise (two logits of this model may be equal) no draft need be right, and a step gives one token at least
        same = next((i for i, (a, b) in enumerate(zip(plain, drafted)) if a != b), len(plain)) - 1  # (the first one is given)
        assert steps <= same // 5 + (30 - same) and same >= 10
    # every token is the best one after those before it, up to what rounding in another batch size may move a logit: hidden rows
    # as in the 16-bit cache (half a step of bf16, 2^-8, about ten times in two layers), and keys and values of two layers that
    # fall to the other side of a border of two codes, by a step of 2^-3 of an element at most
    logits = follow(sd.Model(2, codes=True), drafted[:-1])
    best = logits.max(-1).values
    chosen = logits.gather(1, torch.tensor(drafted[1:], device=logits.device)[:, None])[:, 0]
    assert ((best - chosen) <= (10 * 2.0 ** -8 + 4 * 2.0 ** -3) * logits.std(-1)).all()
