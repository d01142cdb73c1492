"""The mixture-of-experts layer against fp64 within rows_bounds' error bounds: also wide layers
(activations in chunks, passes cut by the results' room), few pairs in either form, many
experts and slots."""
import pytest
import torch

from rows_bounds import LAYERS, layer, layer_inputs, refused
from test_rows_gpu import _need_gpu, bits, check_route  # noqa: F401  (the fixture skips without a GPU)

pytestmark = pytest.mark.gpu

ck = pytest.importorskip("packed_int4_convrot_amd")

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("kind,renormalize", [(torch.float32, True), (torch.bfloat16, False)])
@pytest.mark.parametrize("case", LAYERS)
def test_layer(case, kind, renormalize):
    k = case[4]
    x, logits, tensors = layer_inputs(*case, device=DEV)
    logits = logits.to(kind)
    print("layer", case, flush=True)
    experts = ck.MoeExperts(*tensors)
    out, ids, w = ck.moe(x, logits, experts, k, renormalize)
    check_route(logits, k, renormalize, ids, w)
    assert refused(out, *layer(x, ids, w, tensors)) is None
    assert torch.equal(bits(out), bits(ck.moe_experts(x, ids, w, experts)))
