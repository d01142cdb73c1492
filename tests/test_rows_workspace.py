"""Workspace queries of the mixture-of-experts layer and the adapters (no GPU): 0 for
whatever the entry points refuse."""
import pytest

ck = pytest.importorskip("packed_int4_convrot_amd")
moe, lora = ck.lib.ck_moe_workspace_bytes, ck.lib.ck_lora_workspace_bytes


@pytest.mark.parametrize("T,I,E,k", [(4, 100, 8, 2), (4, 63, 8, 2), (4, 65, 8, 2), (4, 32767, 8, 2)])
def test_moe_workspace_is_zero_for_refused_widths(T, I, E, k):
    assert moe(T, I, E, k) == 0


@pytest.mark.parametrize("M,K,R,L", [(4, 100, 8, 1), (4, 65, 8, 1), (4, 64, 12, 1), (4, 64, 7, 1), (4, 64, 255, 1),
                                     (4, 64, 8, 2 ** 22), (4, 64, 8, 2 ** 40)])
def test_lora_workspace_is_zero_for_refused_sizes(M, K, R, L):
    assert lora(M, K, R, L) == 0


def test_workspaces_of_taken_sizes():
    assert moe(4, 64, 8, 2) > 0 and moe(4, 32768, 1024, 32) > 0
    assert lora(4, 64, 8, 1) > 0 and lora(4, 32768, 256, 2 ** 22 - 1) > 0
