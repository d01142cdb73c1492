"""The adapters against fp64 within rows_bounds' error bounds, without base so that nothing
but their own sum is rounded: every form of the second product at every number of ranks it
is built for."""
import pytest
import torch

from rows_bounds import ADAPTERS, adapter_inputs, adapters, refused
from test_rows_gpu import _need_gpu  # noqa: F401  (the fixture skips without a GPU)

pytestmark = pytest.mark.gpu

ck = pytest.importorskip("packed_int4_convrot_amd")

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("case", ADAPTERS)
def test_adapters(case):
    x, index, tensors = adapter_inputs(*case, device=DEV)
    print("adapters", case, flush=True)
    out = ck.lora_add(x, ck.LoraAdapters(*tensors), index)
    assert refused(out, *adapters(x, index, tensors)) is None
    assert not out[index < 0].any()


@pytest.mark.parametrize("M", [16, 64, 2048])
def test_every_bit_pattern_of_base_is_kept_without_an_adapter(M):
    """Among them NaN with any payload, -0, denormals and infinities."""
    N = max(16, 65536 // M)
    every = torch.arange(65536, dtype=torch.int32, device=DEV).to(torch.int16)
    base = every.repeat(-(-M * N // 65536))[:M * N].view(M, N)
    x = torch.ones((M, 64), device=DEV, dtype=torch.bfloat16)
    handle = ck.LoraAdapters(torch.ones((2, 8, 64), device=DEV, dtype=torch.bfloat16),
                             torch.ones((2, N, 8), device=DEV, dtype=torch.bfloat16))
    for index in ([-1, -1], [-1, 0], [1, -1]):
        index = torch.tensor(index, dtype=torch.int32, device=DEV).repeat(M // 2)
        out = ck.lora_add(x, handle, index, base=base.view(torch.bfloat16)).view(torch.int16)
        assert torch.equal(out[index < 0], base[index < 0])
