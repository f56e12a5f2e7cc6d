"""Expanded latent attention through Serve.prompt against the 64-bit form: both
head shapes, lengths of zero and one and around the steps and row tiles,
more queries than keys, contexts before the queries, no causal mask, rising
scores, values that are not finite where no row may see them, strides and
refusals."""
import numpy as np
import pytest

import serve_case as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from int4_routed_expert_layer_amd import binding as B  # noqa: E402
from int4_routed_expert_layer_amd.serve import Serve  # noqa: E402

DEV = "cuda:0"
TYPE = {"bf16": torch.bfloat16, "f16": torch.float16}
HEADS = {"wide": (192, 256), "narrow": (128, 128)}


class Case:
    def __init__(self, nq, nk, heads, width="wide", dtype="bf16", causal=True, seed=0, scale=0.07, gain=1.0):
        print(f"case nq={nq[:8]} nk={nk[:8]} heads={heads} {width} {dtype} causal={causal} seed={seed}", flush=True)
        g = torch.Generator().manual_seed(2000 + seed)
        self.nq, self.nk, self.heads, self.dtype, self.causal, self.scale = nq, nk, heads, dtype, causal, scale
        self.nope, self.v = HEADS[width]
        dt = TYPE[dtype]
        self.q = (gain * torch.randn(sum(nq), heads, self.nope + 64, generator=g)).to(dt)
        self.kv = torch.randn(sum(nk), heads, self.nope + self.v, generator=g).to(dt)
        self.pe = torch.randn(sum(nk), 64, generator=g).to(dt)
        self.qs = torch.tensor(np.concatenate([[0], np.cumsum(nq)]), dtype=torch.int32)
        self.ks = torch.tensor(np.concatenate([[0], np.cumsum(nk)]), dtype=torch.int32)

    def run(self, **kw):
        s = Serve(self.heads, max(sum(self.nq), 1), len(self.nq), nope=self.nope, v_dim=self.v, dtype=self.dtype)
        out, lse = s.prompt(self.q.to(DEV), self.kv.to(DEV), self.pe.to(DEV), self.qs.to(DEV), self.ks.to(DEV), self.scale, causal=self.causal, return_lse=True, **kw)
        torch.cuda.synchronize()
        assert s.device_errors() == 0
        s.close()
        return out, lse

    def check(self, out, lse, heads=None):
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b, (n, m) in enumerate(zip(self.nq, self.nk)):
            q0, k0 = int(self.qs[b]), int(self.ks[b])
            see = np.tril(np.ones((n, m), bool), m - n) if self.causal else np.ones((n, m), bool)
            for h in heads or range(self.heads):
                q = self.q[q0:q0 + n, h].double().numpy()
                k = np.concatenate([self.kv[k0:k0 + m, h, :self.nope].double().numpy(), self.pe[k0:k0 + m].double().numpy()], 1)
                o, e, bo, be = R.attend(q, k, self.kv[k0:k0 + m, h, self.nope:].double().numpy(), see, self.scale, self.dtype)
                got, gl = out[q0:q0 + n, h], lse[q0:q0 + n, h]
                assert np.all(np.abs(got - o) <= bo), (b, h, np.nanmax(np.abs(got - o) - bo))
                fine = np.isfinite(e)
                assert np.array_equal(np.isneginf(gl), ~fine), (b, h)
                assert np.all(np.abs(gl[fine] - e[fine]) <= be[fine]), (b, h)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("width", ["wide", "narrow"])
def test_lengths_around_steps_and_tiles(width, dtype):
    n = [1, 2, 31, 32, 33, 64, 127, 128, 129, 200, 0, 260]
    c = Case(n, n, 2, width, dtype, seed=1)
    c.check(*c.run())


@pytest.mark.parametrize("width", ["wide", "narrow"])
@pytest.mark.parametrize("causal", [True, False])
def test_contexts_and_queries_without_keys(width, causal):
    """Earlier context, fewer keys than queries (the leading queries see nothing), no keys at all."""
    c = Case([1, 40, 100, 70, 5], [300, 41, 30, 0, 5], 3, width, causal=causal, seed=2)
    out, lse = c.run()
    c.check(out, lse)
    assert torch.all(out[141:211] == 0) and torch.all(torch.isneginf(lse[141:211]))
    if causal:
        assert torch.all(out[41:111] == 0) and torch.all(torch.isneginf(lse[41:111]))


@pytest.mark.parametrize("width", ["wide", "narrow"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scores_that_rise_along_the_keys(width, dtype):
    c = Case([50, 3], [290, 200], 1, width, dtype, seed=3, scale=0.1)
    at = 0
    for m in c.nk:
        ramp = torch.linspace(-3, 3, m)[:, None]
        c.kv[at:at + m, 0, :c.nope] = (0.1 * c.kv[at:at + m, 0, :c.nope].float() + ramp).to(TYPE[dtype])
        at += m
    c.q[..., :c.nope] = (0.1 * c.q[..., :c.nope].float() + 1.0).to(TYPE[dtype])
    c.check(*c.run())


@pytest.mark.parametrize("width", ["wide", "narrow"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_keys_that_a_query_does_not_see_may_hold_anything(width, bad):
    """Key 57 of a causal prompt: its value (one column) and, in the second
    run, its key are not finite.  Earlier queries keep their bits; later ones
    have that column, then everything, not finite."""
    c = Case([130], [130], 2, width, seed=4)
    clean, clean_lse = c.run()
    c.kv[57, 1, c.nope + 9] = bad
    out, lse = c.run()
    assert torch.equal(out[:57], clean[:57]) and torch.equal(out[:, 0], clean[:, 0]) and torch.equal(lse, clean_lse)
    assert not torch.isfinite(out[57:, 1, 9]).any()
    assert torch.equal(out[:, 1, :9], clean[:, 1, :9]) and torch.equal(out[:, 1, 10:], clean[:, 1, 10:])
    c.kv[57, 1, 3] = float("nan")
    out, lse = c.run()
    assert torch.equal(out[:57], clean[:57]) and torch.equal(lse[:57], clean_lse[:57]) and torch.equal(out[:, 0], clean[:, 0])
    assert torch.isnan(out[57:, 1]).all() and torch.isnan(lse[57:, 1]).all()


@pytest.mark.parametrize("width", ["wide", "narrow"])
def test_a_long_prompt_and_the_same_bits_twice(width):
    c = Case([700], [1500], 9, width, seed=5)
    out, lse = c.run()
    again, again_lse = c.run()
    assert torch.equal(out, again) and torch.equal(lse, again_lse)
    c.check(out, lse, heads=[4])


@pytest.mark.parametrize("width", ["wide", "narrow"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,nk", [([40], [2501]), ([1, 300, 5], [1800, 2100, 4]), ([900], [900]), ([1000], [700])])
def test_few_rows_of_many_keys(width, dtype, causal, n, nk):
    """Calls with few tiles, whose keys are divided: parts that some rows or all see, and sequences too short for parts."""
    c = Case(n, nk, 2, width, dtype, causal=causal, seed=11)
    out, lse = c.run()
    c.check(out, lse)
    again, again_lse = c.run()
    assert torch.equal(out, again) and torch.equal(lse, again_lse)


@pytest.mark.parametrize("width", ["wide", "narrow"])
def test_values_that_are_not_finite_in_divided_keys(width):
    """Key 1600 of 1650 is hidden from the first 30 of 80 queries and its value is inf in one column."""
    c = Case([80], [1650], 2, width, seed=12)
    clean, clean_lse = c.run()
    c.kv[1600, 1, c.nope + 9] = float("inf")
    out, lse = c.run()
    assert torch.equal(out[:30], clean[:30]) and torch.equal(out[:, 0], clean[:, 0]) and torch.equal(lse, clean_lse)
    assert not torch.isfinite(out[30:, 1, 9]).any()
    assert torch.equal(out[:, 1, :9], clean[:, 1, :9]) and torch.equal(out[:, 1, 10:], clean[:, 1, 10:])
    c.kv[1600, 1, c.nope + 9] = 0.5
    c.kv[100, 1, 3] = float("nan")                          # a key that all see
    out, lse = c.run()
    assert torch.isnan(out[:, 1]).all() and torch.isnan(lse[:, 1]).all() and torch.equal(lse[:, 0], clean_lse[:, 0])


@pytest.mark.parametrize("width", ["wide", "narrow"])
def test_divided_keys_on_another_stream_and_replayed_from_a_graph(width):
    c = Case([90, 20], [1000, 700], 3, width, seed=13)
    want, want_lse = c.run()
    s = Serve(3, 110, 2, nope=c.nope, v_dim=c.v)
    args = [x.to(DEV) for x in (c.q, c.kv, c.pe, c.qs, c.ks)]
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        s.prompt(*args, c.scale, out=out, lse=lse)
    st.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.prompt(*args, c.scale, out=out, lse=lse)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    s.close()


@pytest.mark.parametrize("width", ["wide", "narrow"])
def test_many_sequences_and_uncovered_tokens(width):
    n = [int(x) for x in np.random.default_rng(6).integers(0, 40, 150)]
    c = Case(n, n, 1, width, seed=6)
    c.check(*c.run())
    c.qs = c.qs.clone()
    c.qs[0] = 3                                             # the first tokens belong to no sequence
    c.ks[0] = 3
    marked = torch.full((sum(n), 1, c.v), 7.0, dtype=torch.bfloat16, device=DEV)
    out, _ = c.run(out=marked)
    assert torch.all(out[:3] == 7.0)


@pytest.mark.parametrize("width", ["wide", "narrow"])
def test_strided_inputs(width):
    c = Case([70, 9], [90, 9], 3, width, seed=7)
    want, want_lse = c.run()
    T, K, d, e = 79, 99, c.nope + 64, c.nope + c.v
    q = torch.full((T, 4, d + 16), float("nan"), dtype=torch.bfloat16, device=DEV)
    q[:, 1:, 8:8 + d] = c.q.to(DEV)
    kv = torch.full((3, K, e), float("nan"), dtype=torch.bfloat16, device=DEV)   # heads outermost
    kv[:] = c.kv.to(DEV).transpose(0, 1)
    pe = torch.full((K, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    pe[:, 64:] = c.pe.to(DEV)
    s = Serve(3, T, 2, nope=c.nope, v_dim=c.v)
    out, lse = s.prompt(q[:, 1:, 8:8 + d], kv.transpose(0, 1), pe[:, 64:], c.qs.to(DEV), c.ks.to(DEV), c.scale, return_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    s.close()


def test_two_parts_joined_by_their_sums():
    """Context and chunk attended apart, joined by lse, are the whole: what the lse output is for."""
    c = Case([33], [140], 4, "narrow", seed=8)
    whole, _ = c.run()
    first, l1 = Case.run(part(c, 0, 107, False))
    second, l2 = Case.run(part(c, 107, 140, True))
    top = torch.maximum(l1, l2)
    a, b = torch.exp(l1 - top)[..., None], torch.exp(l2 - top)[..., None]
    joined = (a * first.float() + b * second.float()) / (a + b)
    big = whole.float().abs().max()
    assert (joined - whole.float()).abs().max() <= 4 * R.UNIT["bf16"] * big    # three roundings of values up to the largest


def part(c, k0, k1, causal):
    d = Case([33], [k1 - k0], 4, "narrow", causal=causal, seed=8)
    d.q, d.kv, d.pe = c.q, c.kv[k0:k1], c.pe[k0:k1]
    return d


def test_bounds_outside_the_call_set_a_flag():
    c = Case([20, 20], [20, 20], 2, seed=9)
    good, _ = c.run()
    s = Serve(2, 40, 2)
    args = [t.to(DEV) for t in (c.q, c.kv, c.pe)]
    for qs, ks in (([0, 20, 41], [0, 20, 40]), ([0, 20, 40], [0, 20, 41]), ([0, 20, 40], [0, -1, 40]), ([0, 20, 10], [0, 20, 40])):
        out = torch.zeros_like(good)
        s.prompt(*args, torch.tensor(qs, dtype=torch.int32, device=DEV), torch.tensor(ks, dtype=torch.int32, device=DEV), c.scale, out=out)
        assert s.device_errors() == 1, (qs, ks)
    s.close()


def test_refusals():
    s = Serve(2, 16, 2)
    q = torch.zeros(8, 2, 256, dtype=torch.bfloat16, device=DEV)
    kv = torch.zeros(8, 2, 448, dtype=torch.bfloat16, device=DEV)
    pe = torch.zeros(8, 64, dtype=torch.bfloat16, device=DEV)
    st = torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    for args in ((q.half(), kv, pe, st, st), (q, kv[..., :440], pe, st, st), (q, kv, pe[:7], st, st), (q, kv, pe, st.long(), st), (q, kv, pe, st, st[:1]), (q[0], kv, pe, st, st)):
        with pytest.raises((TypeError, ValueError)):
            s.prompt(*args, 1.0)
    for scale in (0.0, float("inf")):
        with pytest.raises(B.ColiError) as e:
            s.prompt(q, kv, pe, st, st, scale)
        assert e.value.status == B.E_INVALID
    many = torch.zeros(17, 2, 256, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(B.ColiError):
        s.prompt(many, kv, pe, st, st, 1.0)
    assert s.prompt(q[:0], kv, pe, st * 0, st, 1.0).shape == (0, 2, 256)
    s.close()
