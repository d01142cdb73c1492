"""The bounds of the mixture-of-experts and adapter tests refuse wrong results (no GPU): for
every case of the GPU tests the fp64 definition with a mistake planted in it, and the
correctly rounded result taken."""
import pytest
import torch

from rows_bounds import ADAPTERS, LAYERS, adapter_inputs, adapters, layer, layer_inputs, refused


@pytest.mark.parametrize("case", LAYERS)
def test_mistakes_are_refused(case):
    T, H, I, E, k, _ = case
    x, logits, tensors = layer_inputs(*case)
    v, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, w = ids[:, :k], torch.softmax(v[:, :k].double(), dim=1)
    ref, err = layer(x, ids, w, tensors)
    right = ref.to(torch.bfloat16)
    assert refused(right, ref, err) is None
    assert refused(right + ref.abs().max() * 2.0 ** -9, ref, err) is not None

    def lost(columns):
        t = x.clone()
        t[:, columns] = 0
        return t

    def stale(t, chunk):  # columns from `chunk` on as those before
        t = t.clone()
        t[:, chunk:] = t[:, :t.shape[1] - chunk].clone()
        return t

    w1, s1, z1, w2, s2, z2 = tensors
    first = w.clone()
    first[0, 0] = 0
    wrong = {
        "nothing": torch.zeros_like(right),
        "a tile on": right.roll(16, dims=1),
        "another expert": layer(x, ids, w, tensors, pick=lambda e: (e + 1) % E)[0],
        "h as one bf16": layer(x, ids, w, tensors, hidden=lambda h: h.bfloat16().double())[0],
        "the last group lost": layer(lost(slice(H - 64, H)), ids, w, tensors)[0],
        "one column lost": layer(lost(H - 1), ids, w, tensors)[0],
        "a slot lost": layer(x, ids, first, tensors)[0],
        "gate and up exchanged": layer(x, ids, w, (w1.roll(I, 1), s1.roll(I, 2), None if z1 is None else z1.roll(I, 2),
                                                   w2, s2, z2))[0],
    }
    if z1 is not None:
        wrong["no zeros in the first product"] = layer(x, ids, w, (w1, s1, None, w2, s2, z2))[0]
        wrong["no zeros in the second"] = layer(x, ids, w, (w1, s1, z1, w2, s2, None))[0]
    if T > 1:
        wrong["two tokens exchanged"] = right[[1, 0, *range(2, T)]]
    for width in (4096, 8192):
        if width < H < 2 * width + 64:
            wrong["x's first %d columns again" % width] = layer(stale(x, width), ids, w, tensors)[0]
    if 2048 < I < 4096 + 64:
        wrong["h's first 2048 columns again"] = layer(
            x, ids, w, tensors, hidden=lambda h: torch.cat((h[:, :2048], h[:, :I - 2048]), dim=1))[0]
    for name, bad in wrong.items():
        assert refused(bad.to(torch.bfloat16), ref, err) is not None, name


@pytest.mark.parametrize("case", ADAPTERS)
def test_mistakes_in_adapters_are_refused(case):
    M, K, N, R, L = case
    x, index, tensors = adapter_inputs(*case)
    a, b, scaling, ranks = tensors
    ref, err = adapters(x, index, tensors)
    right = ref.to(torch.bfloat16)
    assert refused(right, ref, err) is None
    lost = x.clone()
    lost[:, K - 1] = 0
    wrong = {
        "nothing": torch.zeros_like(right),
        "a tile on": right.roll(16, dims=1),
        "another adapter": adapters(x, index, tensors, pick=lambda l: (l + 1) % L)[0],
        "A x as one bf16": adapters(x, index, tensors, between=lambda v: v.bfloat16().double())[0],
        "one column lost": adapters(lost, index, tensors)[0],
        "a rank lost": adapters(x, index, (a, b, scaling, ranks - 1))[0],
        "the whole rank": adapters(x, index, (a, b, scaling, torch.full_like(ranks, R)))[0],
        "no scaling": adapters(x, index, (a, b, torch.ones_like(scaling), ranks))[0],
        "every row has one": adapters(x, index.clamp(min=0), tensors)[0],
    }
    if (ranks[index.clamp(min=0).long()][index >= 0] == R).all():
        del wrong["the whole rank"]
    if (index >= 0).all():
        del wrong["every row has one"]
    for name, bad in wrong.items():
        assert refused(bad.to(torch.bfloat16), ref, err) is not None, name
