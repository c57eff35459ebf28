"""The balance loss where the sums of many blocks are joined: one sequence over a cluster of 4 and 8 blocks, some of
them without experts, and more sequences than a warp looks over one by one."""
import pytest
import torch

from test_gpu_balance_loss import built, check, config, inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,pad", [(6400, 256, 4, 0.0), (6400, 130, 4, 0.2), (40000, 256, 8, 0.0), (40000, 256, 8, 0.1),
                                       (40000, 130, 4, 0.1), (40000, 512, 8, 0.3), (20000, 1000, 4, 0.0)])
def test_one_sequence_over_many_blocks(score, T, E, k, pad):
    for dtype in (torch.float32, torch.bfloat16):
        logits, idx, _, mask = inputs(T, E, k, dtype, seed=E, pad=pad)
        check(config(T, E, k, score), logits, idx, None, mask if pad else None, score, torch.full((1,), 1.5, device="cuda"))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,S", [(3000, 8, 1500), (300, 8, 1100), (5000, 64, 200)])
def test_losses_and_gradients_of_many_sequences(score, T, E, S):
    logits, idx, off, mask = inputs(T, E, 2, torch.float32, seqs=S, pad=0.1)
    dloss = torch.rand(S, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") - 0.3
    check(config(T, E, 2, score), logits, idx, off, mask, score, dloss)
