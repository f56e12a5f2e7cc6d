"""Absorbed attention over an 8-bit latent cache (Serve.decode) against the 64-bit form on the values that its rows
stand for: the lengths where steps, waves' shares and pages end, pages smaller than a share, few and many rows,
chains, trees, hidden rows of any bytes, seen NaN, divided contexts, strides, graphs, offsets past 2^31."""
import numpy as np
import pytest

import serve8_case as R8
import serve_case as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from int4_routed_expert_layer_amd import binding as B  # noqa: E402
from int4_routed_expert_layer_amd.serve import Serve  # noqa: E402
from test_gpu_latent_decode import DEV, TYPE, Case, tree  # noqa: E402


class Case8(Case):
    """The same sequences in 8-bit rows; what no row fills is 0xFF: NaN in the values, the rotary part and the scales."""

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        packed = torch.full((*self.cache.shape[:2], R8.ROW8), 0xFF, dtype=torch.uint8)
        for b, n in enumerate(self.lens):
            rows = R8.pack(self.kv[b][:, :R.LATENT].double().numpy(), self.kv[b][:, R.LATENT:], self.dtype) if n else torch.zeros(0, R8.ROW8, dtype=torch.uint8)
            self.kv[b] = torch.from_numpy(R8.unpack(rows, self.dtype)) if n else torch.zeros(0, R.ROW, dtype=torch.float64)
            for i in range(0, n, self.page):
                packed[self.table[b, i // self.page], :len(rows[i:i + self.page])] = rows[i:i + self.page]
        self.cache = packed


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,page", [(1, 16), (5, 8), (16, 64), (33, 32), (64, 4), (128, 1), (40, 2)])
def test_single_tokens_at_the_lengths_where_steps_and_pages_end(dtype, heads, page):
    lens = [1, 2, 7, 8, 9, 31, 32, 33, 63, 64, 65, 127, 200]
    c = Case8(lens, [1] * len(lens), heads, page, dtype, seed=heads)
    c.check(*c.run(), heads=range(0, heads, max(1, heads // 3)))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_chains_of_different_lengths_and_empty_sequences(dtype):
    c = Case8([0, 5, 70, 7, 0, 64, 130, 40], [1, 5, 3, 9, 0, 0, 4, 40], 3, 16, dtype, seed=2)
    out, lse = c.run()
    c.check(out, lse)
    assert torch.all(out[0] == 0) and torch.all(torch.isneginf(lse[0]))
    assert torch.all(torch.isneginf(lse[9:11]))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("nodes,words", [([1, 7, 25], 1), ([64, 63, 2], 1), ([65, 130, 3], 3)])
def test_trees(dtype, nodes, words):
    lens = [n + extra for n, extra in zip(nodes, (0, 40, 95))]
    c = Case8(lens, nodes, 2, 32, dtype, sets=[R.ancestors(tree(n, n)) for n in nodes], words=words, seed=5)
    c.check(*c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads", [2, 64])
def test_what_a_hidden_node_holds_does_not_matter(dtype, heads):
    """Node 2's row is arbitrary bytes, NaN and scales beyond the type among them; node 2 and its child 4 see it."""
    c = Case8([50], [6], heads, 16, dtype, sets=[R.ancestors([-1, 0, 0, 1, 2, 3])], seed=7)
    clean, clean_lse = c.run()
    c.check(clean, clean_lse, heads=[0, heads - 1])
    pos = 50 - 6 + 2
    row = torch.randint(0, 256, (R8.ROW8,), dtype=torch.uint8, generator=torch.Generator().manual_seed(3))
    row[5], row[640:] = 0x7F, 0xFF
    c.cache[c.table[0, pos // 16], pos % 16] = row
    out, lse = c.run()
    for i in (0, 1, 3, 5):
        assert torch.equal(out[i], clean[i]) and torch.equal(lse[i], clean_lse[i]), i


def test_a_nan_that_a_row_sees_spoils_it():
    c = Case8([90], [4], 16, 16, seed=8)
    clean, _ = c.run()
    for pos in (89, 87, 20):
        other = Case8([90], [4], 16, 16, seed=8)
        other.cache[other.table[0, pos // 16], pos % 16, 9] = 0x7F
        out, lse = other.run()
        first = max(0, pos - 86)
        assert torch.equal(out[:first], clean[:first])
        assert torch.isnan(out[first:]).all() and torch.isnan(lse[first:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("down", [False, True])
def test_scores_that_rise_or_fall_along_the_context(dtype, down):
    c = Case8([300], [1], 16, 64, dtype, seed=9)
    ramp = np.linspace(-6, 6, 300)[:, None] * (-1 if down else 1)
    rows = R8.pack(0.2 * c.kv[0][:, :R.LATENT].numpy() + 0.25 * ramp, (0.2 * c.kv[0][:, R.LATENT:] + 0.25 * torch.from_numpy(ramp)).to(TYPE[dtype]), dtype)
    c.kv[0] = torch.from_numpy(R8.unpack(rows, dtype))
    for i in range(0, 300, 64):
        c.cache[c.table[0, i // 64], :len(rows[i:i + 64])] = rows[i:i + 64]
    c.q[:] = (0.1 * c.q.float() + 1.0).to(TYPE[dtype])
    c.check(*c.run())


@pytest.mark.parametrize("lens,nodes,heads", [([5000], [1], 64), ([5000], [1], 16), ([2000, 17, 900, 1], [2, 1, 3, 1], 33), ([150] * 300, [1] * 300, 16), ([700] * 5, [20] * 5, 64)])
def test_split_and_many_sequences(lens, nodes, heads):
    c = Case8(lens, nodes, heads, 32, seed=11)
    out, lse = c.run()
    again, again_lse = c.run()
    assert torch.equal(out, again) and torch.equal(lse, again_lse)
    c.check(out, lse, heads=[0, heads - 1] if sum(nodes) * max(lens) < 200000 else [heads // 2])


@pytest.mark.parametrize("heads", [1, 16, 31, 32, 33, 48])
@pytest.mark.parametrize("bits", [8, 16])
def test_units_of_few_rows_have_the_bits_of_full_ones(heads, bits):
    """A unit of 32 rows or fewer leaves half of the products out; the rows are those of a call with more heads."""
    c = (Case8 if bits == 8 else Case)([700, 45], [1, 1], 64, 16, seed=19)
    want, want_lse = c.run()
    few = (Case8 if bits == 8 else Case)([700, 45], [1, 1], 64, 16, seed=19)
    few.heads, few.q = heads, few.q[:, :heads].contiguous()
    out, lse = few.run()
    assert torch.equal(out, want[:, :heads]) and torch.equal(lse, want_lse[:, :heads])


def test_strided_queries_and_pages_of_an_interleaved_cache():
    c = Case8([77, 20], [2, 1], 6, 16, seed=12)
    want, want_lse = c.run()
    q = torch.zeros(3, 7, R.ROW + 8, dtype=torch.bfloat16, device=DEV)
    q[:, :6, 8:] = c.q.to(DEV)
    layers = torch.full((c.cache.shape[0], 3, 16, R8.ROW8), 0xFF, dtype=torch.uint8, device=DEV)
    layers[:, 1] = c.cache.to(DEV)
    table = torch.full((2, 9), -1, dtype=torch.int32, device=DEV)
    table[:, :c.table.shape[1]] = c.table.to(DEV)
    s = Serve(6, 3, 2, 16)
    s.plan(c.q_start.to(DEV), torch.tensor(c.lens, dtype=torch.int32, device=DEV))
    out, lse = s.decode(q[:, :6, 8:8 + R.LATENT], q[:, :6, 8 + R.LATENT:], layers[:, 1], table[:, :c.table.shape[1]], c.scale, return_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    s.close()


def test_on_another_stream_and_replayed_from_a_graph():
    c = Case8([600, 90], [2, 3], 16, 16, seed=13)
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
            s.plan(starts, lens, n_tok=5)
            assert torch.equal(out, s.decode(ql, qp, cache, table, c.scale))
    s.close()


def test_cache_past_two_to_the_32_bytes():
    page, pages = 64, (1 << 32) // (64 * R8.ROW8) + 600
    c = Case8([150], [1], 16, page, seed=14)
    cache = torch.zeros(pages, page, R8.ROW8, dtype=torch.uint8, device=DEV)
    table = c.table.clone()
    for i in range(table.shape[1]):
        cache[pages - 1 - i] = c.cache[c.table[0, i]].to(DEV)
        table[0, i] = pages - 1 - i
    c.cache, c.table = cache, table
    c.check(*c.run())
    s = Serve(16, 1, 1, page)
    rows = s.read(cache, table.to(DEV), torch.tensor([0, 150], dtype=torch.int32, device=DEV))
    assert np.array_equal(rows.double().cpu().numpy(), c.kv[0].numpy())
    s.close()


@pytest.mark.parametrize("page", [16, 2])
def test_out_of_range_pages_set_flags(page):
    c = Case8([100, 60], [1, 1], 16, page, seed=15)
    good, _ = c.run()
    s = Serve(16, 2, 2, page)
    for at in (0, 48 // page):
        for value in (-1, 1 << 20):
            bad = Case8([100, 60], [1, 1], 16, page, seed=15)
            bad.table[0, at] = value
            out, _ = bad.run(s)
            assert s.device_errors() == 2
            assert torch.equal(out[1], good[1])
    short = Case8([100, 60], [1, 1], 16, page, seed=15)
    short.table = short.table[:, :64 // page].contiguous()
    short.run(s)
    assert s.device_errors() == 2
    s.close()


def test_refusals():
    s = Serve(4, 8, 2, 16)
    q = torch.zeros(2, 4, R.LATENT, dtype=torch.bfloat16, device=DEV)
    p = torch.zeros(2, 4, R.ROPE, dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros(4, 16, R8.ROW8, dtype=torch.uint8, device=DEV)
    table = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    with pytest.raises(B.ColiError) as e:
        s.decode(q, p, cache, table, 1.0)
    assert e.value.status == B.E_STATE
    s.plan(torch.tensor([0, 2], dtype=torch.int32, device=DEV), torch.tensor([9], dtype=torch.int32, device=DEV))
    for bad in (cache[..., :640], cache.view(torch.int8), cache[:, :8], cache.cpu(), cache.transpose(0, 1).contiguous().transpose(0, 1)):
        with pytest.raises((TypeError, ValueError)):
            s.decode(q, p, bad, table, 1.0)
    out = s.decode(q, p, cache, table, 1.0)
    assert torch.all(out == 0)
    s.close()
