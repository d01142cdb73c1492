"""The Python binding of the router, the mixture-of-experts layer and the adapters, without
a GPU: what it hands to the C ABI.  The binding's device checks are replaced so that it takes
CPU tensors, and the entry points by recorders of their arguments."""
import gc

import pytest
import torch

ck = pytest.importorskip("packed_int4_convrot_amd")


@pytest.fixture
def calls(monkeypatch):
    """Arguments of the entry points' calls, which enqueue nothing."""
    seen = []

    def dense(t, name, dtype, shape):
        if not isinstance(t, torch.Tensor) or t.dtype != dtype or tuple(t.shape) != tuple(shape):
            raise ValueError(name)
        return t

    def record(*args):
        seen.append(args)
        return ck.CK_OK
    monkeypatch.setattr(ck, "_dense", dense)
    monkeypatch.setattr(ck, "_stream", lambda t: 0)
    for name in ("ck_lora_add", "ck_moe_experts_w4a16"):
        monkeypatch.setattr(ck.lib, name, record)
    return seen


def adapter_tensors():
    return [torch.ones((2, 8, 64), dtype=torch.bfloat16), torch.ones((2, 16, 8), dtype=torch.bfloat16),
            torch.ones((2,)), torch.ones((2,), dtype=torch.int32)]


def expert_tensors():
    return [torch.ones((2, 128, 32), dtype=torch.uint8), torch.ones((2, 1, 128), dtype=torch.bfloat16),
            torch.ones((2, 1, 128), dtype=torch.bfloat16), torch.ones((2, 64, 32), dtype=torch.uint8),
            torch.ones((2, 1, 64), dtype=torch.bfloat16), torch.ones((2, 1, 64), dtype=torch.bfloat16)]


def lora_call(handle):
    ck.lora_add(torch.ones((3, 64), dtype=torch.bfloat16), handle, torch.zeros((3,), dtype=torch.int32))


def moe_call(handle):
    ck.moe_experts(torch.ones((3, 64), dtype=torch.bfloat16), torch.zeros((3, 2), dtype=torch.int32),
                   torch.ones((3, 2)), handle)


HANDLES = [(ck.LoraAdapters, adapter_tensors, lora_call, slice(7, 11)),
           (ck.MoeExperts, expert_tensors, moe_call, slice(10, 16))]


@pytest.mark.parametrize("kind,tensors,call,at", HANDLES)
def test_a_handle_holds_the_memory_whose_address_it_passes(calls, kind, tensors, call, at):
    """Putting other storage into the caller's tensors frees nothing that a later call reads."""
    mine = tensors()
    held = [t.untyped_storage()._weak_ref() for t in mine]
    handle = kind(*mine)
    where = [t.data_ptr() for t in mine]
    call(handle)
    assert list(calls[-1][at]) == where
    for t in mine:
        t.data = torch.zeros((4,), dtype=t.dtype)
    del mine, t
    gc.collect()
    assert not any(torch.UntypedStorage._expired(w) for w in held)
    call(handle)
    assert list(calls[-1][at]) == where == [t.data_ptr() for t in handle.tensors]
    for w in held:
        torch.UntypedStorage._free_weak_ref(w)


@pytest.mark.parametrize("kind,tensors,call,at", HANDLES)
def test_a_handle_whose_storage_was_given_up_is_refused(calls, kind, tensors, call, at):
    for i in range(len(tensors())):
        mine = tensors()
        handle = kind(*mine)
        mine[i].untyped_storage().resize_(0)
        with pytest.raises(ValueError):
            call(handle)
    assert not calls


@pytest.mark.parametrize("kind,tensors,call,at", HANDLES)
def test_values_written_into_a_handles_tensors_count(kind, tensors, call, at, calls):
    mine = tensors()
    handle = kind(*mine)
    for t in mine:
        t.fill_(3)
    assert all((t == 3).all() for t in handle.tensors)


NOT_MATRICES = [None, 3.0, [[1.0] * 64] * 3, torch.ones(()), torch.ones((64,), dtype=torch.bfloat16),
                torch.ones((1, 3, 64), dtype=torch.bfloat16)]


@pytest.mark.parametrize("bad", NOT_MATRICES)
def test_what_is_not_a_matrix_is_refused(calls, monkeypatch, bad):
    adapters, experts = ck.LoraAdapters(*adapter_tensors()), ck.MoeExperts(*expert_tensors())
    monkeypatch.setattr(ck, "_LOGIT_KIND", {})
    x, index = torch.ones((3, 64), dtype=torch.bfloat16), torch.zeros((3,), dtype=torch.int32)
    ids, weights = torch.zeros((3, 2), dtype=torch.int32), torch.ones((3, 2))
    for call in (lambda: ck.lora_add(bad, adapters, index), lambda: ck.lora_add(x, adapters, bad),
                 lambda: ck.moe_experts(bad, ids, weights, experts), lambda: ck.moe_experts(x, bad, weights, experts),
                 lambda: ck.moe_experts(x, ids, bad, experts), lambda: ck.moe_route(bad, 2),
                 lambda: ck.moe(x, bad, experts, 2)):
        with pytest.raises(ValueError):
            call()
    if bad is not None:
        for call in (lambda: ck.lora_add(x, adapters, index, base=bad), lambda: ck.lora_add(x, adapters, index, out=bad),
                     lambda: ck.lora_add(x, adapters, index, workspace=bad),
                     lambda: ck.moe_experts(x, ids, weights, experts, out=bad),
                     lambda: ck.moe_experts(x, ids, weights, experts, workspace=bad)):
            with pytest.raises(ValueError):
                call()
    assert not calls


@pytest.mark.parametrize("k", [0, -1, -2 ** 40, 2 ** 31, 2 ** 32 + 2])
def test_slot_counts_outside_an_int32_are_refused(k):
    with pytest.raises(ValueError):
        ck._slots(None, None, 0, k, torch.device("cpu"))
