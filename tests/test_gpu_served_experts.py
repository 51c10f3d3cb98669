"""A served expert layer's prompts: the same choices as its decoding steps, and the same bits every time."""
import math

import pytest
import torch

import tiled_dense_gemm_relu_amd as gr
from tiled_dense_gemm_relu_amd.expert_layer import ExpertLayer, ServedExperts

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def served():
    return ServedExperts(ExpertLayer(8, 128, 256, seed=5), 4)


def inputs(tokens, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(tokens, 128, generator=g, device=DEV).bfloat16(), torch.randn(tokens, 8, generator=g, device=DEV)


def test_prompts_repeat_themselves(served):
    x, logits = inputs(700)
    want = served.prompt(x, logits)
    for _ in range(20):
        assert torch.equal(served.prompt(x, logits), want)


def test_prompts_choose_as_decoding_does(served):
    x, logits = inputs(60)
    logits[0] = 0.5                                      # ties: the lowest indices
    logits[1, 2:] = -math.inf                            # two experts to choose from
    logits[2] = -math.inf                                # none
    logits[3, 5], logits[4, 6] = math.nan, math.inf      # no order
    logits[5] = logits[5].round()
    decoded, prompt = served.decode(x, logits).float(), served.prompt(x, logits).float()
    assert not decoded[2].any() and not prompt[2].any()
    for t in (3, 4):
        assert decoded[t].isnan().all() and prompt[t].isnan().all()
    for t in set(range(60)) - {2, 3, 4}:
        # another expert's outputs are unrelated; those of rows and hidden values in 8 bits are off by half a step
        # of e4m3 (2^-4) of each at most, twice
        assert float((decoded[t] - prompt[t]).norm() / decoded[t].norm()) <= 2 * 2.0 ** -4, t


def test_an_expert_that_is_never_chosen_may_hold_anything():
    layer = ExpertLayer(4, 128, 128, seed=6)
    layer.weights[1][3] = float("nan")
    served = ServedExperts(layer, 3)
    x, logits = inputs(40, 2)
    logits = logits[:, :4].contiguous()
    logits[:, 3] = -math.inf
    logits[::2, 2] = -math.inf                           # fewer than three to choose from
    assert served.decode(x, logits).isfinite().all() and served.prompt(x, logits).isfinite().all()


def test_no_tokens_one_token_and_too_many_choices(served):
    x, logits = inputs(3)
    assert served.prompt(x[:0], logits[:0]).shape == (0, 128)
    # (products of other sizes may take other kernels, whose sums differ in fp32: a rounding to bf16 and to e4m3 can turn)
    one = served.prompt(x[:1], logits[:1]).float()
    assert float((one - served.prompt(x, logits)[:1].float()).norm() / one.norm()) <= 2.0 ** -5
    for top in (0, 9):
        with pytest.raises(ValueError, match="top"):
            ServedExperts(ExpertLayer(8, 128, 256, seed=5), top)
