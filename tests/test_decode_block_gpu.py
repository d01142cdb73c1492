"""The example's decode step on a GPU: each operator's result from the step's own
inputs against the 64-bit definition, and the captured step replayed on new inputs
against the same calls one by one."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 7, 40])
def test_decode_block(tokens):
    import packed_int4_convrot_amd as ck
    from decode_block import DecodeBlock
    from test_rows_gpu import assert_within, ref_experts, ref_lora

    print("decode block of %d tokens" % tokens, flush=True)
    block = DecodeBlock(tokens, 256, 192, 16, 3, 4, 8, seed=tokens)
    graph = block.capture()
    g = torch.Generator(device="cuda:0").manual_seed(tokens)
    for _ in range(3):
        block.x.normal_(generator=g)
        block.index.random_(-1, 4, generator=g)
        out = block.step().clone()
        y, ids, weights = block.y.clone(), block.ids.clone(), block.weights.clone()

        base = ck.linear(block.x, 64, 8, *block.projection[:2], True)
        assert_within(y, *ref_lora(block.x, *block.adapters.tensors, block.index, base))
        logits = block.logits.double()
        assert torch.equal(ids.long(), logits.sort(dim=1, descending=True, stable=True).indices[:, :3])
        assert ((weights - logits.gather(1, ids.long()).softmax(dim=1)).abs() < 1e-5).all()
        assert_within(out, *ref_experts(y, ids, weights, block.experts.tensors))

        block.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(block.out, out) and torch.equal(block.y, y) and torch.equal(block.ids, ids)
