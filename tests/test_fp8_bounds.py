"""The bounds of the 8-bit float tests refuse wrong results (no GPU): the fp64 definitions with
a mistake planted in them, and the correctly rounded result taken."""
import pytest
import torch

import fp8_bounds as ref
from fp8_bounds import random_rows, random_weight, refused


def rounded(y):
    return y.to(torch.bfloat16)


def all_refused(wrong, right):
    for name, bad in wrong.items():
        assert refused(rounded(bad), *right) is not None, name


@pytest.mark.parametrize("M,K,N", [(1, 16, 16), (5, 144, 48), (3, 1024, 272), (33, 400, 144), (130, 256, 384), (2, 8320, 32)])
def test_mistakes_in_a_linear_are_refused(M, K, N):
    x, (codes, scales) = random_rows(M, K, M + K + N).double(), random_weight(N, K, N)
    w = ref.weight(codes, scales)
    bias = torch.randn((N,), generator=torch.Generator().manual_seed(1)).bfloat16().double()
    right = ref.linear(x, w, bias)
    assert refused(rounded(right[0]), *right) is None
    q, s = ref.quant(x)
    exact = lambda a, v=w: a @ v.t() + bias  # noqa: E731
    lost = x.clone()
    lost[:, K - 1] = 0
    wrong = {"nothing": torch.zeros_like(right[0]), "no bias": right[0] - bias, "x not quantised": exact(x),
             "another scale in the last block": exact(ref.values(q, torch.cat((s[:, :-1], 2 * s[:, -1:]), dim=1))),
             "the last column lost": exact(ref.values(*ref.quant(lost)))}
    if K > 128:
        wrong["the first block's scale for all"] = exact(q * s[:, :1])
    for name, axis in (("a block on", 1), ("a row of blocks on", 0)):
        moved = scales.view(torch.uint8).roll(1, axis)
        if not torch.equal(moved, scales.view(torch.uint8)):
            wrong["weight scales " + name] = exact(ref.values(q, s), ref.weight(codes, moved.view(scales.dtype)))
    if N > 32:
        wrong["a tile on"] = right[0].roll(32, dims=1)
    if M > 1:
        wrong["two rows exchanged"] = right[0][[1, 0, *range(2, M)]]
    all_refused(wrong, right)


def block(M, H, I, seed=0):
    x = 0.25 * random_rows(M, H, M + H + I + seed).double()
    c1, s1 = random_weight(2 * I, H, H + seed)
    w1 = ref.weight(c1, s1) * 2.0 ** -round(0.5 * torch.tensor(float(H)).log2().item())
    return x, w1, ref.weight(*random_weight(H, I, I + seed))


@pytest.mark.parametrize("M,H,I", [(3, 144, 256), (17, 512, 384), (65, 400, 128), (40, 64, 1152)])
def test_mistakes_in_a_feed_forward_block_are_refused(M, H, I):
    x, w1, w2 = block(M, H, I)
    right, kept = ref.ffn(x, w1, w2)
    assert refused(rounded(right[0]), *right) is None and refused(rounded(kept[0]), *kept) is None
    other = w1.roll(I, 0)
    wrong = {"nothing": torch.zeros_like(right[0]), "gate and up exchanged": ref.ffn(x, other, w2)[0][0],
             "h a column on": ref.ffn(x, w1, w2, hidden=lambda h: h.roll(1, dims=1))[0][0],
             "h of 32 columns lost": ref.ffn(x, w1, w2, hidden=lambda h: torch.cat((h[:, :-32], 0 * h[:, -32:]), dim=1))[0][0],
             "h in three bits": ref.ffn(x, w1, w2, hidden=lambda h: torch.ldexp(torch.round(torch.frexp(h)[0] * 8) / 8, torch.frexp(h)[1]))[0][0],
             "no activation": ref.product(ref.values(*ref.quant(kept[0][:, :I] * kept[0][:, I:])), w2)[0]}
    all_refused(wrong, right)
    all_refused({"exchanged": kept[0].roll(I, 1), "a tile on": kept[0].roll(32, 1)}, kept)


@pytest.mark.parametrize("M,H,I", [(3, 144, 256), (17, 512, 384), (65, 400, 128), (40, 64, 1152)])
def test_mistakes_in_a_backward_pass_are_refused(M, H, I):
    _, w1, w2 = block(M, H, I)
    dy = 2.0 ** -10 * random_rows(M, H, M).double()
    gu = (2 * torch.randn((M, 2 * I), generator=torch.Generator().manual_seed(M + I))).bfloat16().double()
    right = ref.backward(dy, gu, w1, w2)
    assert refused(rounded(right[0]), *right) is None
    change = lambda f: ref.backward(dy, gu, w1, w2, change=f)[0]  # noqa: E731
    g, u = gu[:, :I], gu[:, I:]
    s = torch.sigmoid(g)
    dh = ref.values(*ref.quant(dy)) @ w2
    wrong = {"nothing": torch.zeros_like(right[0]), "exchanged": change(lambda dg, du: (du, dg)),
             "no gradient of the gate": change(lambda dg, du: (0 * dg, du)), "of up": change(lambda dg, du: (dg, 0 * du)),
             "32 columns lost": change(lambda dg, du: (torch.cat((dg[:, :-32], 0 * dg[:, -32:]), dim=1), du)),
             "the logistic function's slope left out": change(lambda dg, du: (dh * u * s, du)),
             "the other sign of it": change(lambda dg, du: (dh * u * s * (1 - g * (1 - s)), du)),
             "two rows exchanged": right[0][[1, 0, *range(2, M)]]}
    all_refused(wrong, right)


def test_the_quantiser_of_the_definitions():
    """Against a table of all e4m3 values, and scales by counting up."""
    table = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double()
    table = table[table.isfinite()].sort().values.unique()
    v = torch.cat((table, (table[1:] + table[:-1]) / 2, torch.randn((4000,), generator=torch.Generator().manual_seed(0)).double() * 60))
    v = v.clamp(-448, 448)
    got = ref.e4m3(v)
    near = (v[:, None] - table).abs()
    assert ((got - v).abs() == near.min(dim=1).values).all()
    tie = (near == near.min(dim=1, keepdim=True).values).sum(dim=1) == 2
    even = got[tie].float().to(torch.float8_e4m3fn).view(torch.uint8) % 2 == 0
    assert tie.sum() > 200 and even.all()
    for a in (2.0 ** -133, 1e-30, 1.0, 1.75, 1.7500001, 447.9, 448.0, 448.1, 1e30):
        s = float(ref.scale_of(torch.tensor([a], dtype=torch.float64)))
        assert a <= 448 * s and (a > 448 * s / 2 or s == 2.0 ** -127)
    assert float(ref.scale_of(torch.zeros(1, dtype=torch.float64))) == 1.0
