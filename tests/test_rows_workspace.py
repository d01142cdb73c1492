"""Workspace queries of the mixture-of-experts layer and the adapters (no GPU): 0 for
whatever the entry points refuse, and enough for every smaller call too."""
import os
import shutil
import subprocess

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


@pytest.mark.parametrize("K,R,L", [(64, 8, 1), (3840, 16, 32), (3840, 64, 8), (10240, 40, 7), (3840, 256, 300)])
def test_a_lora_workspace_serves_every_smaller_call(K, R, L):
    rows = list(range(1, 2200)) + list(range(2200, 40000, 61)) + [2 ** 22 - 1]
    sizes = [lora(M, K, R, L) for M in rows]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    for M in (1, 63, 64, 65, 301, 1024, 1025, 8192, 10000, 20000):
        assert lora(M, K, R, L) <= lora(M, K + 64, R, L) and lora(M, K, 8, L) <= lora(M, K, R, L)
        assert lora(M, K, R, 1) <= lora(M, K, R, L) and lora(M, K, R, 2 ** 20) <= lora(M, K, R, L)


@pytest.mark.parametrize("I,E,k", [(64, 8, 1), (64, 8, 7), (1280, 64, 8), (128, 1024, 32)])
def test_a_layer_workspace_serves_every_smaller_call(I, E, k):
    sizes = [moe(T, I, E, k) for T in list(range(1, 1200)) + [2 ** 22 - 1]]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.skipif(not shutil.which("g++"), reason="host compiler g++ not found")
def test_the_parts_of_every_size_fit_the_room(tmp_path):
    """lora_splits() * M rows against lora_room_rows(), over the sizes' whole range."""
    here = os.path.dirname(os.path.abspath(__file__))
    exe = str(tmp_path / "rows_room")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", os.path.join(here, "sanitize", "rows_room.cpp"),
                    "-o", exe], check=True, timeout=120)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "fit" in r.stdout, r.stdout
