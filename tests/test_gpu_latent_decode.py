"""Absorbed latent attention through Serve.decode against the 64-bit form:
lengths of zero and one, tiles and pages that end inside a step, odd heads,
chains and trees of one and more mask words, rows that see nothing, values that
are not finite where nothing may see them, rising scores, split contexts,
strides, streams, graphs and a cache past 2^31 elements."""
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


class Case:
    """Sequences of `lens` cached positions and `nodes` tokens of this step."""

    def __init__(self, lens, nodes, heads, page=16, dtype="bf16", sets=None, words=1, seed=0, scale=1 / 16, gain=1.0, fill=float("nan"), spare=2):
        print(f"case lens={lens[:8]} nodes={nodes[:8]} heads={heads} page={page} {dtype} words={words} seed={seed}", flush=True)
        g = torch.Generator().manual_seed(1000 + seed)
        self.lens, self.nodes, self.heads, self.page, self.dtype, self.sets, self.scale = lens, nodes, heads, page, dtype, sets, scale
        dt, T = TYPE[dtype], sum(nodes)
        each = [-(-n // page) for n in lens]
        order = torch.randperm(sum(each) + spare, generator=g).tolist()
        table = torch.full((len(lens), max(max(each), 1)), -1, dtype=torch.int32)
        self.cache = torch.full((len(order), page, R.ROW), fill, dtype=dt)
        self.kv = []
        at = 0
        for b, n in enumerate(lens):
            rows = torch.randn(n, R.ROW, generator=g).to(dt)
            self.kv.append(rows)
            for i in range(each[b]):
                table[b, i] = order[at + i]
                part = rows[i * page:(i + 1) * page]
                self.cache[order[at + i], :len(part)] = part
            at += each[b]
        self.table = table
        self.q = (gain * torch.randn(T, heads, R.ROW, generator=g)).to(dt)
        self.q_start = torch.tensor(np.concatenate([[0], np.cumsum(nodes)]), dtype=torch.int32)
        self.mask = None if sets is None else torch.from_numpy(np.concatenate([R.words_of(s, words) for s in sets]))
        self.words = words

    def seen(self, b):
        sets = self.sets
        if sets is not None:
            sets = [{d for d in s if d < 64 * self.words} for s in sets[b]]
        return R.visible(self.nodes[b], self.lens[b], sets)

    def run(self, serve=None, **kw):
        own = serve is None
        if own:
            serve = Serve(self.heads, max(sum(self.nodes), 1), len(self.lens), self.page, dtype=self.dtype)
        q = self.q.to(DEV)
        serve.plan(self.q_start.to(DEV), torch.tensor(self.lens, dtype=torch.int32, device=DEV))
        out, lse = serve.decode(q[..., :R.LATENT].contiguous(), q[..., R.LATENT:].contiguous(), self.cache.to(DEV), self.table.to(DEV), self.scale,
                                tree_mask=None if self.mask is None else self.mask.to(DEV), return_lse=True, **kw)
        torch.cuda.synchronize()
        if own:
            assert serve.device_errors() == 0
            serve.close()
        return out, lse

    def check(self, out, lse, heads=None):
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        q0 = 0
        for b, n in enumerate(self.nodes):
            kv = self.kv[b].double().numpy()
            see = self.seen(b)
            for h in heads or range(self.heads):
                q = self.q[q0:q0 + n, h].double().numpy()
                o, e, bo, be = R.attend(q, kv, kv[:, :R.LATENT], see, self.scale, self.dtype)
                got, gl = out[q0:q0 + n, h], lse[q0:q0 + n, h]
                assert np.all(np.abs(got - o) <= bo), (b, h, np.nanmax(np.abs(got - o) - bo))
                fine = np.isfinite(e)
                assert np.array_equal(np.isneginf(gl), ~fine), (b, h)
                assert np.all(np.abs(gl[fine] - e[fine]) <= be[fine]), (b, h)
            q0 += n


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,page", [(1, 16), (5, 8), (16, 64), (64, 4), (128, 1)])
def test_single_tokens_at_the_lengths_where_steps_and_pages_end(dtype, heads, page):
    lens = [1, 2, 31, 32, 33, 63, 64, 65, 127, 200]
    c = Case(lens, [1] * len(lens), heads, page, dtype, seed=heads)
    c.check(*c.run(), heads=range(0, heads, max(1, heads // 3)))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_chains_of_different_lengths_and_empty_sequences(dtype):
    c = Case([0, 5, 70, 7, 0, 64, 130, 40], [1, 5, 3, 9, 0, 0, 4, 40], 3, 16, dtype, seed=2)
    out, lse = c.run()
    c.check(out, lse)
    assert torch.all(out[0] == 0) and torch.all(torch.isneginf(lse[0]))      # nothing cached
    assert torch.all(torch.isneginf(lse[9:11]))                               # nine tokens, seven cached: two see nothing


def tree(n, seed):
    r = np.random.default_rng(seed)
    return [-1] + [int(r.integers(max(0, j - 5), j)) for j in range(1, n)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("nodes,words", [([1, 7, 25], 1), ([64, 63, 2], 1), ([65, 130, 3], 3), ([70, 9], 1)])
def test_trees(dtype, nodes, words):
    lens = [n + extra for n, extra in zip(nodes, (0, 40, 95))]
    sets = [R.ancestors(tree(n, n)) for n in nodes]
    c = Case(lens, nodes, 2, 32, dtype, sets=sets, words=words, seed=5)
    c.check(*c.run())


def test_a_node_that_sees_nothing():
    c = Case([3, 40], [3, 4], 2, 16, sets=[[{0}, set(), {0, 2}], [set(), {1}, set(), {0, 3}]], seed=6)
    out, lse = c.run()
    c.check(out, lse)
    assert torch.all(out[1] == 0) and torch.all(torch.isneginf(lse[1]))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("heads", [2, 64])
def test_what_a_hidden_node_holds_does_not_matter(bad, heads):
    """Node 2's row is not finite; only node 2 and its child 4 see it."""
    parents = [-1, 0, 0, 1, 2, 3]
    c = Case([50], [6], heads, 16, sets=[R.ancestors(parents)], seed=7)
    clean, clean_lse = c.run()
    c.check(clean, clean_lse, heads=[0, heads - 1])
    pos = 50 - 6 + 2
    c.cache[c.table[0, pos // 16], pos % 16, 3:200:7] = bad
    out, lse = c.run()
    for i in range(6):
        if i in (2, 4):
            if bad != bad:
                assert torch.isnan(out[i]).all() and torch.isnan(lse[i]).all()
        else:
            assert torch.equal(out[i], clean[i]) and torch.equal(lse[i], clean_lse[i]), i


def test_chain_hides_later_tokens_that_are_not_finite():
    c = Case([90], [4], 16, 16, seed=8)
    clean, _ = c.run()
    pos = 89
    c.cache[c.table[0, pos // 16], pos % 16] = float("nan")
    out, _ = c.run()
    assert torch.equal(out[:3], clean[:3]) and torch.isnan(out[3]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("down", [False, True])
def test_scores_that_rise_or_fall_along_the_context(dtype, down):
    """Each step exceeds (or falls short of) the one before by far more than the slack of the running maximum."""
    c = Case([300], [1], 16, 64, dtype, seed=9)
    ramp = torch.linspace(-6, 6, 300)[:, None] * (-1 if down else 1)
    c.kv[0][:] = (0.2 * c.kv[0].float() + 0.25 * ramp).to(TYPE[dtype])
    for i in range(-(-300 // 64)):
        part = c.kv[0][i * 64:(i + 1) * 64]
        c.cache[c.table[0, i], :len(part)] = part
    c.q[:] = (0.1 * c.q.float() + 1.0).to(TYPE[dtype])       # scores from about -54 to 54
    c.check(*c.run())


@pytest.mark.parametrize("lens,nodes,heads", [([5000], [1], 64), ([2000, 17, 900, 1], [2, 1, 3, 1], 33), ([150] * 300, [1] * 300, 16), ([700] * 5, [20] * 5, 64)])
def test_split_and_many_sequences(lens, nodes, heads):
    c = Case(lens, nodes, heads, 32, seed=11)
    out, lse = c.run()
    again, again_lse = c.run()
    assert torch.equal(out, again) and torch.equal(lse, again_lse)            # the same bits every time
    c.nodes, keep = nodes, nodes
    heads_checked = [0, heads - 1] if sum(nodes) * max(lens) < 200000 else [heads // 2]
    c.check(out, lse, heads=heads_checked)
    assert c.nodes is keep


def test_strided_queries_and_pages_of_an_interleaved_cache():
    """Queries as slices of one projection, the cache as one layer of [pages, layers, rows]."""
    c = Case([77, 20], [2, 1], 6, 16, seed=12)
    want, want_lse = c.run()
    q = torch.zeros(3, 7, R.ROW + 8, dtype=torch.bfloat16, device=DEV)
    q[:, :6, 8:] = c.q.to(DEV)
    layers = torch.full((c.cache.shape[0], 3, 16, R.ROW), float("nan"), dtype=torch.bfloat16, device=DEV)
    layers[:, 1] = c.cache.to(DEV)
    table = torch.full((2, 9), -1, dtype=torch.int32, device=DEV)
    table[:, :c.table.shape[1]] = c.table.to(DEV)
    s = Serve(6, 3, 2, 16)
    s.plan(c.q_start.to(DEV), torch.tensor(c.lens, dtype=torch.int32, device=DEV))
    out, lse = s.decode(q[:, :6, 8:8 + R.LATENT], q[:, :6, 8 + R.LATENT:], layers[:, 1], table[:, :c.table.shape[1]], c.scale, return_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    s.close()


@pytest.mark.parametrize("longest,heads", [(150, 16), (900, 65)])
def test_more_sequences_than_a_workgroup_has_threads(longest, heads):
    """1100 sequences, some of them empty: the plan takes them in turns."""
    lens = [int(x) for x in np.random.default_rng(21).integers(0, longest, 1100)]
    c = Case(lens, [min(n, 1) for n in lens], heads, 64, seed=21)
    c.check(*c.run(), heads=[heads // 2])


def test_on_another_stream_and_replayed_from_a_graph():
    c = Case([600, 90], [2, 3], 16, 16, seed=13)
    want, want_lse = c.run()
    s = Serve(16, 5, 2, 16)
    q, cache, table = c.q.to(DEV), c.cache.to(DEV), c.table.to(DEV)
    ql, qp = q[..., :R.LATENT].contiguous(), q[..., R.LATENT:].contiguous()
    starts, lens = c.q_start.to(DEV), torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        s.plan(starts, lens, n_tok=5)
        s.decode(ql, qp, cache, table, c.scale, out=out, lse=lse)
    st.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.plan(starts, lens, n_tok=5)
        s.decode(ql, qp, cache, table, c.scale, out=out, lse=lse)
    for length in (600, 333, 600):
        lens[0] = length
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        if length == 600:
            assert torch.equal(out, want) and torch.equal(lse, want_lse)
        else:
            short = Case([600, 90], [2, 3], 16, 16, seed=13)
            short.lens = [333, 90]
            short.kv[0] = short.kv[0][:333]
            eager, _ = short.run()
            assert torch.equal(out, eager)
    s.close()


def test_cache_past_two_to_the_31_elements():
    page, pages = 64, (1 << 31) // (64 * R.ROW) + 600
    c = Case([150], [1], 16, page, seed=14)
    cache = torch.zeros(pages, page, R.ROW, dtype=torch.bfloat16, device=DEV)
    table = c.table.clone()
    for i in range(table.shape[1]):
        cache[pages - 1 - i] = c.cache[c.table[0, i]].nan_to_num().to(DEV)
        table[0, i] = pages - 1 - i
    c.cache, c.table = cache, table
    c.check(*c.run())


def test_out_of_range_pages_and_bounds_set_flags():
    c = Case([100, 60], [1, 1], 16, 16, seed=15, fill=0.0)
    good, _ = c.run()
    s = Serve(16, 2, 2, 16)
    for value in (-1, 1 << 20):
        c.table[0, 3] = value
        out, _ = c.run(s)
        assert s.device_errors() == 2
        assert torch.equal(out[1], good[1])
    short = Case([100, 60], [1, 1], 16, 16, seed=15, fill=0.0)
    short.table = short.table[:, :4].contiguous()           # 64 of 100 positions have a page
    out, _ = short.run(s)
    assert s.device_errors() == 2
    for starts in ([0, 2, 1], [0, -1, 2], [0, 1, 3]):
        s.plan(torch.tensor(starts, dtype=torch.int32, device=DEV), torch.tensor([5, 5], dtype=torch.int32, device=DEV), n_tok=2)
        assert s.device_errors() == 1
    s.plan(torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV), torch.tensor([5, -1], dtype=torch.int32, device=DEV), n_tok=2)
    assert s.device_errors() == 1
    s.close()


def test_refusals():
    s = Serve(4, 8, 2, 16)
    q = torch.zeros(2, 4, R.LATENT, dtype=torch.bfloat16, device=DEV)
    p = torch.zeros(2, 4, R.ROPE, dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros(4, 16, R.ROW, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    starts, lens = torch.tensor([0, 2], dtype=torch.int32, device=DEV), torch.tensor([9], dtype=torch.int32, device=DEV)
    with pytest.raises(B.ColiError) as e:
        s.decode(q, p, cache, table, 1.0)
    assert e.value.status == B.E_STATE
    assert B.lib.coli_latent_decode(s.handle, None, 0, 0, None, 0, 0, None, 0, 0, None, 0, 0, None, 0, 1.0, 0, None, None, None) == B.E_STATE
    with pytest.raises(B.ColiError):
        s.plan(starts, lens, n_tok=9)
    s.plan(starts, lens)
    for bad in (dict(scale=0.0), dict(scale=float("nan")), dict(scale=-1.0)):
        with pytest.raises(B.ColiError) as e:
            s.decode(q, p, cache, table, **bad)
        assert e.value.status == B.E_INVALID
    for args in ((q.half(), p, cache, table), (q.cpu(), p, cache, table), (q[:1], p, cache, table), (q, p[..., :32], cache, table),
                 (q, p, cache[:, :8], table), (q, p, cache.transpose(0, 1).contiguous().transpose(0, 1), table), (q, p, cache, table.long()),
                 (q.transpose(1, 2).contiguous().transpose(1, 2), p, cache, table), (None, p, cache, table)):
        with pytest.raises((TypeError, ValueError)):
            s.decode(*args, 1.0)
    odd = torch.zeros(2 * 4 * R.LATENT + 1, dtype=torch.bfloat16, device=DEV)[1:].view(2, 4, R.LATENT)
    with pytest.raises(B.ColiError) as e:
        s.decode(odd, p, cache, table, 1.0)
    assert e.value.status == B.E_INVALID and "aligned" in str(e.value)
    with pytest.raises(ValueError):
        s.decode(q, p, cache, table, 1.0, tree_mask=torch.zeros(2, 0, dtype=torch.int64, device=DEV)[:1])
    out = s.decode(q, p, cache, table, 1.0)
    assert out.shape == (2, 4, R.LATENT)
    s.close()
    with pytest.raises(ValueError):
        s.plan(starts, lens, n_tok=2)
