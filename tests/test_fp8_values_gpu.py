"""What is not finite, and what is nearly so, in the 8-bit float operators' weights, rows and gates."""
import pytest
import torch

import fp8_bounds as ref
from fp8_bounds import random_rows, random_weight, refused
from test_fp8_gpu import DEV, NAN, bits, block, ck, same

pytestmark = pytest.mark.gpu

INF = float("inf")
# One row, a few from bf16 and from codes, tiles, K split; K inside a block and of 17 blocks.
ROWS = [(1, 272), (3, 272), (20, 272), (20, 2160), (100, 272), (100, 2160), (700, 272)]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def spoiled(got, clean, columns):
    """NaN in `columns` of every row, the clean result's bits in all others."""
    keep = torch.ones(got.shape[1], dtype=torch.bool, device=DEV)
    keep[columns] = False
    assert clean.isfinite().all()
    assert got[:, columns].isnan().all() and same(got[:, keep], clean[:, keep])


def linears(x, codes, scales):
    """From rows and from codes."""
    weights = ck.Fp8Weights(codes, scales)
    return ck.fp8_linear(x, weights), ck.fp8_gemm(*ck.fp8_quant(x), weights)


@pytest.mark.parametrize("M,K", ROWS)
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_not_finite_in_a_weight_spoils_its_block(bad, M, K):
    N = 400
    g = torch.Generator().manual_seed(K)
    w = (torch.randn((N, K), generator=g) * K ** -0.5).bfloat16().to(DEV)
    w[140] = 0                                      # in the block's rows
    x, dy = random_rows(M, K, 2, DEV), random_rows(M, N, 3, DEV)
    codes, scales = ck.fp8_quantize_weights(w)
    clean = linears(x, codes, scales)
    clean_t = linears(dy, *ck.Fp8Weights(codes, scales).transposed().tensors)
    w[150, 131] = bad
    codes_bad, scales_bad = ck.fp8_quantize_weights(w)
    want = bits(scales).clone()
    want[1, 1] = 255
    assert torch.equal(bits(scales_bad), want)
    for got, good in zip(linears(x, codes_bad, scales_bad), clean):
        spoiled(got, good, slice(128, 256))
    for got, good in zip(linears(dy, *ck.Fp8Weights(codes_bad, scales_bad).transposed().tensors), clean_t):
        spoiled(got, good, slice(128, 256))


@pytest.mark.parametrize("M,K", ROWS)
def test_nan_among_given_codes_and_scales(M, K):
    """Weights made elsewhere: a NaN code spoils its own output, a NaN scale its block's."""
    N = 400
    x, (codes, scales) = random_rows(M, K, 2, DEV), random_weight(N, K, 4, DEV)
    codes.view(torch.uint8)[130] = 0
    clean = linears(x, codes, scales)
    sick = codes.clone()
    sick.view(torch.uint8)[150, 131] = 0x7f
    for got, good in zip(linears(x, sick, scales), clean):
        spoiled(got, good, [150])
    sick = scales.clone()
    sick.view(torch.uint8)[1, 0] = 255
    for got, good in zip(linears(x, codes, sick), clean):
        spoiled(got, good, slice(128, 256))


@pytest.mark.parametrize("M", [1, 3, 40, 90, 700])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("column", [5, 384 + 5])
def test_a_gate_or_up_that_is_not_finite_spoils_its_row(M, bad, column):
    H, I = 272, 384
    x, w1, w2 = block(M, H, I)
    x[0, 0] = 1                                     # no row of zeros there
    back = ck.Fp8Ffn(*w1, *w2).transposed()
    gate_up = torch.randn((M, 2 * I), generator=torch.Generator().manual_seed(M)).bfloat16().to(DEV)
    clean = ck.fp8_ffn_backward(x, gate_up, back)
    gate_up[0, column] = bad
    dx = ck.fp8_ffn_backward(x, gate_up, back)
    assert clean.isfinite().all() and dx[0].isnan().all() and same(dx[1:], clean[1:])


@pytest.mark.parametrize("M,K", ROWS)
def test_the_largest_rows_whose_codes_stay_below_2_to_128(M, K):
    """x up to 1.9296875 2^127, whose code stands for 1.875 2^127 (from 1.9375 2^127 on it would be 2^128),
    against weights whose products are of ordinary size."""
    x, (codes, scales) = random_rows(M, K, 5, DEV), random_weight(144, K, 6, DEV)
    x = (x.sign() * torch.full_like(x, 1.9296875) * 2.0 ** 127).bfloat16()
    small = (scales.view(torch.uint8).int() - 100).to(torch.uint8).view(ck.E8M0)
    want = ref.linear(x.double(), ref.weight(codes, small))
    for out in linears(x, codes, small):
        assert out.isfinite().all() and refused(out, *want) is None
