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
