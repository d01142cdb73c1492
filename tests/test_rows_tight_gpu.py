"""The mixture-of-experts layer against fp64 within rows_bounds' error bounds: wide layers
(activations in chunks, passes cut by the results' room), few pairs in either form, many
experts and slots, weights beyond 32-bit offsets, activations near the sums' range."""
import pytest
import torch

from rows_bounds import LAYERS, expert_weights, layer, layer_inputs, refused
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


@pytest.mark.parametrize("T,I", [(2, 1280), (12, 2112)])
def test_weights_beyond_32_bit_offsets(T, I):
    """Few and many pairs: the last experts of slabs of more than 4 GiB, all of it distinct
    weights, give the bits that the same experts give by themselves."""
    E, H, k = 1024, 4096, 2
    g = torch.Generator(device=DEV).manual_seed(I)

    def one(N, K):
        p = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device=DEV, generator=g)
        s = torch.empty((E, K // 64, N), dtype=torch.bfloat16, device=DEV).uniform_(0.002, 0.02, generator=g)
        z = torch.empty((E, K // 64, N), dtype=torch.bfloat16, device=DEV).normal_(0, 0.01, generator=g)
        return p, s, z
    big = one(2 * I, H) + one(H, I)
    assert big[0].numel() > 2 ** 32 and big[3].numel() > 2 ** 31 and (I < 2112 or big[3].numel() > 2 ** 32)
    print("offsets T=%d I=%d" % (T, I), flush=True)
    first = E - 3
    small = [t[first:].clone() for t in big]
    x = torch.randn((T, H), device=DEV, generator=g).bfloat16()
    ids = torch.stack((torch.arange(T, device=DEV) % 3, (torch.arange(T, device=DEV) + 1) % 3), dim=1).int()
    w = torch.rand((T, k), device=DEV, generator=g)
    out = ck.moe_experts(x, ids + first, w, ck.MoeExperts(*big))
    assert torch.equal(bits(out), bits(ck.moe_experts(x, ids, w, ck.MoeExperts(*small))))
    assert refused(out, *layer(x, ids, w, small)) is None


@pytest.mark.parametrize("T", [2, 12])
def test_activations_near_the_range_of_the_sums(T):
    """|x| just below 3.7e34, of which 64 products with codes up to 143 stay finite."""
    H, I, E, k = 256, 128, 4, 2
    tensors = expert_weights(E, H, I, True, seed=T)
    for i in (1, 2):
        tensors[i] = (tensors[i].double() * 2.0 ** -118).bfloat16()
    g = torch.Generator().manual_seed(T)
    x = (torch.randn((T, H), generator=g).sign() * torch.empty((T, H)).uniform_(3e34, 3.69e34, generator=g)).bfloat16()
    x[:, :64] = x[:, :64].abs()  # a group whose sum is as large as can be
    assert x.abs().max() < 3.7e34
    tensors = [t.to(DEV) for t in tensors]
    x, logits = x.to(DEV), torch.randn((T, E), generator=g).to(DEV)
    out, ids, w = ck.moe(x, logits, ck.MoeExperts(*tensors), k)
    assert out.isfinite().all() and refused(out, *layer(x, ids, w, tensors)) is None
