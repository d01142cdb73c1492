"""The layer's ids and weights are those of the router alone, bit for bit, whichever of its
forms a call takes."""
import pytest
import torch

from test_rows_gpu import _need_gpu, expert_weights  # noqa: F401  (the fixture skips without a GPU)

pytestmark = pytest.mark.gpu

ck = pytest.importorskip("packed_int4_convrot_amd")

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("E", [5, 32, 64, 100, 128, 200, 256, 300, 1024])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renormalize", [True, False])
def test_layer_routes_as_the_router(E, kind, renormalize):
    H, I, k = 64, 64, 2
    experts = ck.MoeExperts(*expert_weights(E, H, I, False, seed=E))
    g = torch.Generator(device=DEV).manual_seed(E)
    for T in (1, 8, 9):  # up to 16 pairs a workgroup routes its own token
        for _ in range(8):
            logits = (torch.randn((T, E), device=DEV, generator=g) * 2).to(kind)
            x = torch.randn((T, H), device=DEV, generator=g).bfloat16()
            _, ids, w = ck.moe(x, logits, experts, k, renormalize)
            rids, rw = ck.moe_route(logits, k, renormalize)
            assert torch.equal(ids, rids) and torch.equal(w, rw), (T, (w - rw).abs().max())
