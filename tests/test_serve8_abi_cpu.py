"""Checks of the 8-bit cache, shared prefixes and beam search that need no GPU: NULL handles are refused before a device
is touched, and the 64-bit forms that the GPU tests compare with agree with elementary special cases."""
import numpy as np
import torch

import serve8_case as R8
from int4_routed_expert_layer_amd import binding as B


def test_null_handles():
    assert B.lib.coli_latent8_append(None, None, 0, None, 0.0, None, None, 0, 0, None, None, 0, None, 0, 0, None, 0, 0, None, None) == B.E_INVALID
    assert B.lib.coli_latent8_decode(None, None, 0, 0, None, 0, 0, None, 0, 0, None, 0, 0, None, 0, 1.0, 0, None, None, None) == B.E_INVALID
    assert B.lib.coli_latent8_keep(None, None, 0, 0, 0, 0, None, 0, 0, None, None, 0, 0, None, 0, 0, None) == B.E_INVALID
    assert B.lib.coli_latent_read(None, 0, None, 0, 0, None, 0, 0, None, None, 0, 0, None, 0, None) == B.E_INVALID
    assert B.lib.coli_latent_plan_shared(None, None, None, 0, 0, None, None, 0, None) == B.E_INVALID
    assert B.lib.coli_beam_select(None, None, 0, 0, 1, None, 0, 1, 1, None, None, None, None) == B.E_INVALID
    assert B.lib.coli_beam_reorder(None, 0, None, 0, 0, 0, 0, None, 0, 0, None, None, 0, 1, None, 0, None) == B.E_INVALID
    assert b"handle" in B.lib.coli_serve_last_error(None)


def test_e4m3_values_and_codes():
    v = R8.VALUES
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0x38] == 1 and v[0x7E] == 448 and np.isnan(v[0x7F]) and v[0xB8] == -1
    fine = ~np.isnan(v)
    assert np.array_equal(torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()[fine], v[fine])
    x = np.random.default_rng(0).standard_normal(5000) * 2.0 ** np.random.default_rng(1).integers(-11, 7, 5000)
    assert np.array_equal(R8.codes(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    half = np.array([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 440.0])   # ties go to the even value
    assert np.array_equal(v[R8.codes(half)], [16, 20, 0, 2.0 ** -8, 448.0])


def test_scales_and_rows():
    for dtype in ("bf16", "f16"):
        most = np.array([0.0, 448.0, 448.0001, 224.0, 2.0 ** -15 * 448, 1e-30, 60000.0])
        k = R8.exponents(most, dtype)
        assert k[1] == 0 and k[2] == 1 and k[3] == -1 and k[0] == R8.LEAST[dtype]
        assert np.all(most <= 448 * 2.0 ** k.astype(float) + (k == R8.MOST[dtype]) * 1e9)
        x = np.random.default_rng(2).standard_normal((3, 512))
        rope = torch.randn(3, 64).to(R8.TYPE[dtype])
        rows = R8.pack(x, rope, dtype)
        assert rows.shape == (3, R8.ROW8) and rows.dtype == torch.uint8
        y = R8.unpack(rows, dtype)
        assert np.array_equal(y[:, 512:], rope.double().numpy())
        R8.check_rows(rows, x, dtype)
        assert np.array_equal(R8.unpack(R8.pack(y[:, :512], rope, dtype), dtype), y)                     # what is representable stays
        assert np.array_equal(torch.from_numpy(y).to(R8.TYPE[dtype]).double().numpy(), y)                # and is of the 16-bit type


def test_selection_form():
    logits, scores = np.log(np.array([[[0.5, 0.25, 0.25], [0.9, 0.1, 0.0]]]) + 1e-300), np.log(np.array([[0.6, 0.4]]))
    s, p, t = R8.select(logits, scores, 4)
    assert p.tolist() == [[1, 0, 0, 0]] and t.tolist() == [[0, 0, 1, 2]]
    assert np.allclose(np.exp(s), [[0.36, 0.3, 0.15, 0.15]])
    s, p, t = R8.select(np.zeros((1, 2, 2)), np.array([[0.0, -np.inf]]), 3)
    assert p.tolist() == [[0, 0, -1]] and t.tolist() == [[0, 1, -1]] and np.isneginf(s[0, 2])


def test_reordering_form():
    cache = torch.arange(6 * 2).view(1, 6, 2, 1)
    table = torch.tensor([[0, 1], [0, 2], [0, 3]], dtype=torch.int32)
    new, t = R8.reorder(cache, table, [3], np.array([[1, 1, 1]]), 2)
    assert t.tolist() == [[0, 2], [0, 1], [0, 3]]             # place 0 keeps beam 1's page, the others take over those of 0 and 2
    assert new[0, 1, 0] == new[0, 3, 0] == cache[0, 2, 0] and new[0, 1, 1] == cache[0, 1, 1]
    same, t = R8.reorder(cache, table, [3], np.array([[0, -1, 2]]), 2)
    assert torch.equal(same, cache) and torch.equal(t, table)
