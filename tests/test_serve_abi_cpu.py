"""Host-side checks of the serving operators that need no GPU: sizes and NULL
arguments are refused before a device is touched, the allocation cap covers
the handle, and the 64-bit forms that the GPU tests compare with agree with
elementary special cases."""
import ctypes as C

import numpy as np
import pytest

import serve_case as R
from int4_routed_expert_layer_amd import binding as B
from int4_routed_expert_layer_amd.serve import ServeDims

GOOD = dict(n_heads=64, latent=512, rope=64, nope=192, v_dim=256, page_size=64, max_tokens=128, max_seqs=8, half=0)


def create(**kw):
    d = ServeDims(**{**GOOD, **kw})
    h = C.c_void_p()
    st = B.lib.coli_serve_create(C.byref(d), 0, C.byref(h))
    if st == B.OK:
        B.lib.coli_serve_destroy(h)
    else:
        assert not h
    return st


@pytest.mark.parametrize("kw", [dict(n_heads=0), dict(max_tokens=0), dict(max_seqs=-1), dict(page_size=0), dict(page_size=48), dict(page_size=1 << 17), dict(half=2)])
def test_invalid_sizes(kw):
    assert create(**kw) == B.E_INVALID
    assert B.lib.coli_serve_last_error(None)


@pytest.mark.parametrize("kw", [dict(latent=256), dict(rope=32), dict(nope=64), dict(nope=128), dict(v_dim=128), dict(n_heads=2000),
                                dict(max_tokens=1 << 30), dict(max_seqs=1 << 21)])
def test_unsupported_sizes(kw):
    assert create(**kw) == B.E_UNSUPPORTED


def test_null_arguments():
    h = C.c_void_p()
    assert B.lib.coli_serve_create(None, 0, C.byref(h)) == B.E_INVALID
    assert B.lib.coli_serve_create(C.byref(ServeDims(**GOOD)), 0, None) == B.E_INVALID
    assert B.lib.coli_serve_destroy(None) == B.OK
    assert B.lib.coli_serve_device_errors(None, None) == B.E_INVALID
    assert B.lib.coli_latent_plan(None, None, None, 0, 0, None) == B.E_INVALID
    assert B.lib.coli_latent_decode(None, None, 0, 0, None, 0, 0, None, 0, 0, None, 0, 0, None, 0, 1.0, 0, None, None, None) == B.E_INVALID
    assert B.lib.coli_latent_prompt(None, None, 0, 0, None, 0, 0, None, 0, None, None, 0, 0, 0, 0, 1.0, None, None, None) == B.E_INVALID
    assert B.lib.coli_latent_append(None, None, 0, None, 0.0, None, None, 0, 0, None, None, 0, None, 0, 0, None, 0, 0, None, None) == B.E_INVALID
    assert B.lib.coli_latent_keep(None, None, 0, 0, 0, 0, None, 0, 0, None, None, 0, 0, None, 0, 0, None) == B.E_INVALID
    assert B.lib.coli_draft_verify(None, None, 0, None, 0, 0, 1, None, None, None, 0, 0, None, None, 0, None, 1, None, None, None) == B.E_INVALID
    assert b"handle" in B.lib.coli_serve_last_error(None)


def test_the_allocation_cap_covers_the_handle():
    B.set_alloc_limit(1 << 20)
    try:
        assert create() == B.E_NOMEM
    finally:
        B.set_alloc_limit(-1)


def test_a_device_that_is_not_there():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert create() == B.E_DEVICE


def test_attention_form_special_cases():
    r = np.random.default_rng(0)
    k, v, q = r.standard_normal((9, 16)), r.standard_normal((9, 5)), r.standard_normal((2, 16))
    see = np.ones((2, 9), bool)
    out, lse, _, _ = R.attend(0 * q, k, v, see, 1.0, "bf16")
    assert np.allclose(out, v.mean(0)) and np.allclose(lse, np.log(9))        # equal scores: the mean
    see[1] = False
    see[1, 4] = True
    out, lse, _, _ = R.attend(q, k, v, see, 0.5, "bf16")
    assert np.allclose(out[1], v[4]) and np.isclose(lse[1], 0.5 * q[1] @ k[4])  # one key: its value
    see[1] = False
    out, lse, _, _ = R.attend(q, k, v, see, 0.5, "bf16")
    assert np.all(out[1] == 0) and np.isneginf(lse[1])


def test_visibility_forms():
    chain = R.visible(3, 5)
    assert chain.tolist() == [[True] * 3 + [False] * 2, [True] * 4 + [False], [True] * 5]
    sets = R.ancestors([-1, 0, 0, 1])
    assert sets == [{0}, {0, 1}, {0, 2}, {0, 1, 3}]
    assert np.array_equal(R.visible(3, 5, R.ancestors([-1, 0, 1])), chain)    # a chain as a tree
    assert R.words_of([{0, 63, 64}], 1)[0, 0] == -2 ** 63 + 1
    assert R.visible(4, 2).sum() == 3                                         # fewer positions than tokens


def test_rotation_keeps_lengths_and_norm_scales():
    r = np.random.default_rng(1)
    x = r.standard_normal((4, 64))
    a = r.uniform(0, 6, (4, 32))
    for inter in (True, False):
        y = R.rotate(x, np.cos(a), np.sin(a), inter)
        assert np.allclose((y ** 2).sum(1), (x ** 2).sum(1))
        assert np.allclose(R.rotate(y, np.cos(a), -np.sin(a), inter), x)
    rows = R.norm_rows(5 * r.standard_normal((3, 576)), np.ones(512), 0.0, np.ones((3, 32)), np.zeros((3, 32)), True)
    assert np.allclose((rows[:, :512] ** 2).mean(1), 1)


def test_verify_form_draws_from_the_target():
    """Exhaustively over a fine grid of u: the first token's probability is the
    target's, for a refused-and-resampled draft and for two children."""
    p = np.array([[0.5, 0.3, 0.2]] * 3)
    q = np.array([[0.2, 0.6, 0.2]] * 3)
    us = (np.arange(4000) + 0.5) / 4000
    got = np.zeros(3)
    for x in range(3):
        for u in us:
            path, nxt, _ = R.verify(p[:2], q[:2], [0, x], [-1, 0], [0, u], np.ones(3), 9)
            if len(path) == 2:
                got[x] += q[0, x] / 4000
            else:
                r = np.maximum(p[0] - q[0], 0)
                got += q[0, x] / 4000 * r / r.sum()
    assert np.allclose(got, p[0], atol=1e-3)
    got = np.zeros(3)
    for u1 in us[::20]:
        for u2 in us[::20]:
            path, _, _ = R.verify(p, None, [0, 0, 1], [-1, 0, 0], [0, u1, u2], np.ones(3), 9)
            if len(path) == 2:
                got[[0, 1][path[1] - 1]] += 1 / 200 ** 2
            else:
                got[2] += 1 / 200 ** 2
    assert np.allclose(got, p[0], atol=1e-2)
