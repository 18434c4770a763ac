"""The decode-step operators together (examples/speculative_decode.py): what is decoded with drafted trees is what the
model decodes one token at a time."""
import os
import sys

import pytest
import torch

from mixture_experts_ffn_moe_gb300 import build

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def follow(model, tokens):
    """Logits after every token, one at a time."""
    dev, rows = model.device, []
    one = torch.ones(1, dtype=torch.int64, device=dev)
    for i, t in enumerate(tokens):
        rows.append(model.step(torch.tensor([t], device=dev), torch.zeros(1, dtype=torch.int64, device=dev), one, i)[0])
    return torch.stack(rows)


@pytest.mark.parametrize("hit", [0.0, 0.7, 1.0])
def test_drafted_decoding_takes_the_models_best_tokens(hit):
    import speculative_decode as sd
    plain, steps = sd.generate(sd.Model(), 7, 40)
    assert steps == 40
    drafted, steps = sd.generate(sd.Model(), 7, 40, known=plain, hit=hit, seed=3)
    assert steps <= 40 and (hit < 1.0 or steps <= 16)  # five tokens a step where the draft is always right
    # every token is the best one after those before it, up to what rounding in another batch size may move a logit:
    # the hidden rows are bf16 (half a step 2^-8 each of about ten times in two layers, of rows of norm 1)
    logits = follow(sd.Model(), drafted[:-1])
    best = logits.max(-1).values
    chosen = logits.gather(1, torch.tensor(drafted[1:], device=logits.device)[:, None])[:, 0]
    spread = logits.std(-1)
    assert ((best - chosen) <= 10 * 2.0 ** -8 * 4 * spread).all()


def test_sampled_decoding_with_drafts_is_reproducible():
    import speculative_decode as sd
    plain, _ = sd.generate(sd.Model(1), 3, 20, temperature=0.7, seed=5)
    a, _ = sd.generate(sd.Model(1), 3, 20, known=plain, temperature=0.7, seed=6)
    b, _ = sd.generate(sd.Model(1), 3, 20, known=plain, temperature=0.7, seed=6)
    assert a == b and len(a) == 21
