"""Absorbed attention of groups that share a prefix (Serve.plan with group_start and prefix_len) against the 64-bit
form over each sequence's whole context: prefixes of every length, groups of uneven sequences, empty and single ones,
sequences of no group, both kinds of cache, chains and trees, hidden and seen NaN, plans that do not fit, graphs,
flags and refusals."""
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


def ints(a):
    return torch.as_tensor(np.ascontiguousarray(a)).to(DEV, torch.int32)


class Shared(Case):
    """groups: (prefix, [own length per sequence], [tokens per sequence]); a prefix of None: sequences of no group.
    The own length counts what lies behind the prefix, the step's tokens among it."""

    def __init__(self, groups, heads, page=16, dtype="bf16", bits=16, trees=False, seed=0, copies=False):
        print(f"groups={[(p, o[:4]) for p, o, _ in groups][:4]} heads={heads} page={page} {dtype} bits={bits} seed={seed}", flush=True)
        g = torch.Generator().manual_seed(500 + seed)
        self.heads, self.page, self.dtype, self.scale, self.bits, self.words = heads, page, dtype, 1 / 16, bits, 1
        dt, pages, self.kv, tables, self.lens, self.nodes = TYPE[dtype], [], [], [], [], []
        width = R.ROW if bits == 16 else R8.ROW8

        def rows(n):
            x = torch.randn(n, R.ROW, generator=g).to(dt)
            return x if bits == 16 else R8.pack(x[:, :R.LATENT].double().numpy(), x[:, R.LATENT:], dtype)

        def paged(r, at):
            """Pages of rows r, the first of them at a page's row `at`."""
            out = []
            for i in range(0, at + len(r), page):
                p = torch.full((page, width), float("nan"), dtype=dt) if bits == 16 else torch.full((page, width), 0xFF, dtype=torch.uint8)
                lo, hi = max(i, at), min(i + page, at + len(r))
                p[lo - i:hi - i] = r[lo - at:hi - at]
                out.append(len(pages))
                pages.append(p)
            return out

        self.starts, self.prefixes = [], []
        for prefix, own, nodes in groups:
            head = rows(prefix or 0)
            whole = (prefix or 0) // page * page
            first = paged(head[:whole], 0) if whole else []
            if prefix is not None:
                self.starts.append(len(self.lens))
                self.prefixes.append(prefix)
            for o, n in zip(own, nodes):
                behind = rows(o)
                tables.append((paged(head[:whole], 0) if copies and whole else first) + paged(torch.cat([head[whole:], behind]), 0))
                full = torch.cat([head, behind])
                self.kv.append(full.double() if bits == 16 else torch.from_numpy(R8.unpack(full, dtype)) if len(full) else torch.zeros(0, R.ROW).double())
                self.lens.append(len(full))
                self.nodes.append(n)
            if prefix is not None:
                self.end = len(self.lens)
        self.starts.append(self.end)
        order = torch.randperm(len(pages), generator=g)
        self.cache = torch.stack(pages)[torch.argsort(order)]
        self.table = torch.full((len(tables), max(1, max(map(len, tables)))), -1, dtype=torch.int32)
        for b, t in enumerate(tables):
            self.table[b, :len(t)] = order[t]
        T = sum(self.nodes)
        self.q = torch.randn(T, heads, R.ROW, generator=g).to(dt)
        self.q_start = torch.tensor(np.concatenate([[0], np.cumsum(self.nodes)]), dtype=torch.int32)
        self.sets = [R.ancestors(tree(n, n)) if n else [] for n in self.nodes] if trees else None
        self.mask = torch.from_numpy(np.concatenate([R.words_of(s, 1) for s in self.sets])) if trees else None

    def run(self, serve=None, share=True, flags=0, prefixes=None, starts=None):
        own = serve is None
        if own:
            serve = Serve(self.heads, max(sum(self.nodes), 1), len(self.lens), self.page, dtype=self.dtype)
        q = self.q.to(DEV)
        more = dict(group_start=ints(starts or self.starts), prefix_len=ints(prefixes or self.prefixes)) if share else {}
        serve.plan(self.q_start.to(DEV), ints(self.lens), **more)
        out, lse = serve.decode(q[..., :R.LATENT].contiguous(), q[..., R.LATENT:].contiguous(), self.cache.to(DEV), self.table.to(DEV), self.scale,
                                tree_mask=None if self.mask is None else self.mask.to(DEV), return_lse=True)
        torch.cuda.synchronize()
        assert serve.device_errors() == flags
        if own:
            serve.close()
        return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("heads", [1, 5, 16, 64])
@pytest.mark.parametrize("prefix", [0, 1, 63, 64, 65, 127, 128, 200])
def test_prefixes_where_tiles_and_pages_end(prefix, heads, bits, dtype):
    c = Shared([(prefix, [1, 2, 33, 64, 65], [1] * 5)], heads, 16, dtype, bits, seed=prefix + heads)
    c.check(*c.run(), heads=sorted({0, heads // 2, heads - 1}))


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("heads,page", [(3, 64), (16, 1), (33, 32), (40, 16)])
def test_uneven_groups_beside_others(heads, page, bits):
    """Groups of one, of two with an empty sequence, of many; sequences of no group before, between and behind."""
    c = Shared([(None, [70, 0, 5], [1, 0, 2]), (300, [4, 150, 9, 1], [3, 1, 2, 1]), (130, [20], [2]), (None, [], []), (100, [7, 0, 40], [1, 0, 1]), (64, [1] * 9, [1] * 9)], heads, page, "bf16", bits, seed=heads)
    # the middle group of no sequences and one whose sequences are those of no group
    c.check(*c.run(), heads=[0, heads - 1])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bits", [16, 8])
def test_chains_and_trees_behind_a_prefix(bits, dtype):
    c = Shared([(200, [30, 9, 64], [5, 9, 25]), (90, [12, 3], [12, 3])], 3, 16, dtype, bits, trees=True, seed=3)
    c.check(*c.run())
    c = Shared([(200, [30, 9, 64], [5, 9, 25]), (90, [12, 3], [12, 3])], 64, 16, dtype, bits, seed=4)
    c.check(*c.run(), heads=[0, 63])


def test_a_prefix_that_is_not_all_context_is_shared_as_far_as_it_is():
    """prefix_len beyond the context of the shortest sequence, beyond every sequence, below zero."""
    c = Shared([(200, [1, 30, 80], [1, 20, 60])], 16, 16, seed=5)
    want, want_lse = c.run()
    c.check(want, want_lse, heads=[0, 15])
    c = Shared([(100, [40, 30, 90], [1, 1, 1])], 16, 16, seed=6)
    c.check(*c.run(prefixes=[100]), heads=[0, 15])
    for prefix in (-5, 0, 63):
        got, lse = c.run(prefixes=[prefix])
        plain, plain_lse = c.run(share=False)
        assert torch.equal(got, plain) and torch.equal(lse, plain_lse)


@pytest.mark.parametrize("bits", [16, 8])
def test_the_prefix_is_read_once(bits):
    """Of all but the first sequence the table has no pages for the prefix's whole tiles."""
    c = Shared([(256, [10, 20, 30], [1, 1, 1])], 16, 64, "bf16", bits, seed=7)
    want, want_lse = c.run()
    c.check(want, want_lse, heads=[3])
    c.table[1:, :4] = -1
    out, lse = c.run()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    copies = Shared([(256, [10, 20, 30], [1, 1, 1])], 16, 64, "bf16", bits, seed=7, copies=True)
    copies.check(*copies.run(), heads=[3])


def test_the_first_sequence_of_a_group_may_have_no_tokens():
    c = Shared([(256, [0, 20, 30], [0, 1, 1])], 16, 64, seed=8)
    want, want_lse = c.run()
    c.check(want, want_lse, heads=[3])
    c.table[0] = -1
    out, lse = c.run()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("bits", [16, 8])
def test_divided_prefixes_and_repeated_bits(bits):
    c = Shared([(5000, [1, 300, 70], [1, 1, 2]), (3000, [40] * 6, [1] * 6)], 24, 32, "bf16", bits, seed=9)
    out, lse = c.run()
    again, again_lse = c.run()
    assert torch.equal(out, again) and torch.equal(lse, again_lse)
    c.check(out, lse, heads=[0, 23])


@pytest.mark.parametrize("n,heads", [(600, 64), (1100, 4), (200, 16), (64, 128)])
def test_many_sequences_whether_their_pieces_fit_or_not(n, heads):
    """600 units and 600 more of the prefix do not fit, nor do 1100 sequences."""
    c = Shared([(70, [1 + i % 3 for i in range(n)], [1] * n)], heads, 16, seed=10)
    c.check(*c.run(), heads=[heads // 2])


def test_what_is_not_finite():
    c = Shared([(128, [10, 20], [2, 1]), (64, [3, 3], [1, 1])], 16, 16, seed=11)
    clean, _ = c.run()
    bad = Shared([(128, [10, 20], [2, 1]), (64, [3, 3], [1, 1])], 16, 16, seed=11)
    bad.cache[bad.table[0, 1], 3, 9] = float("nan")           # of the first group's prefix
    out, lse = bad.run()
    assert torch.isnan(out[:3]).all() and torch.isnan(lse[:3]).all() and torch.equal(out[3:], clean[3:])
    bad = Shared([(128, [10, 20], [2, 1]), (64, [3, 3], [1, 1])], 16, 16, seed=11)
    pos = 128 + 10 - 1                                        # token 1 of sequence 0, hidden from token 0
    bad.cache[bad.table[0, pos // 16], pos % 16, 9] = float("nan")
    out, _ = bad.run()
    assert torch.equal(out[0], clean[0]) and torch.isnan(out[1]).all() and torch.equal(out[2:], clean[2:])


def test_captured_and_replayed_with_other_lengths():
    c = Shared([(300, [30, 9, 64], [1, 1, 1]), (150, [12, 3], [1, 1])], 16, 16, seed=12)
    want, want_lse = c.run()
    s = Serve(16, 5, 5, 16)
    q, cache, table = c.q.to(DEV), c.cache.to(DEV), c.table.to(DEV)
    ql, qp = q[..., :R.LATENT].contiguous(), q[..., R.LATENT:].contiguous()
    q_start, lens, starts, prefix = c.q_start.to(DEV), ints(c.lens), ints(c.starts), ints(c.prefixes)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.plan(q_start, lens, n_tok=5, group_start=starts, prefix_len=prefix)
        s.decode(ql, qp, cache, table, c.scale, out=out, lse=lse)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.plan(q_start, lens, n_tok=5, group_start=starts, prefix_len=prefix)
        s.decode(ql, qp, cache, table, c.scale, out=out, lse=lse)
    for cut, share in ((0, 300), (20, 300), (0, 64), (0, 0), (0, 300)):
        lens[0] = c.lens[0] - cut
        prefix[0] = share
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert s.device_errors() == 0
        got, got_lse = out.clone(), lse.clone()
        other = Shared([(300, [30, 9, 64], [1, 1, 1]), (150, [12, 3], [1, 1])], 16, 16, seed=12)
        other.lens[0] -= cut
        other.kv[0] = other.kv[0][:other.lens[0]]
        other.check(got, got_lse, heads=[0, 15])
        if (cut, share) == (0, 300):
            assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
    s.close()


def test_a_plan_without_groups_after_one_with():
    c = Shared([(300, [30, 9], [1, 1])], 16, 16, seed=13)
    plain = c.run(share=False)
    s = Serve(16, 2, 2, 16)
    for share in (True, False, True, False):
        out, lse = c.run(s, share=share)
        c.check(out, lse, heads=[7])
        if not share:
            assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])
    s.close()


@pytest.mark.parametrize("starts", [[0, 3, 2], [-1, 2, 4], [0, 2, 5], [3, 1, 4]])
def test_groups_out_of_order_set_a_flag_and_are_not_shared(starts):
    c = Shared([(130, [30, 9], [1, 1]), (130, [5, 6], [1, 1])], 16, 16, seed=14)
    out, lse = c.run(starts=starts, flags=1)
    plain, plain_lse = c.run(share=False)
    assert torch.equal(out, plain) and torch.equal(lse, plain_lse)


def test_a_sequence_out_of_bounds_leaves_its_group_unshared():
    """The bad sequence's own result is unspecified; the others' are right, in its group and elsewhere."""
    c = Shared([(130, [30, 9, 8], [1, 1, 1]), (130, [5, 6], [1, 1])], 16, 16, seed=15)
    want, _ = c.run()
    lens = list(c.lens)
    lens[1] = -4
    c.lens = lens
    out, _ = c.run(flags=1)
    keep = [0, 2, 3, 4]
    c.lens[1] = 139
    plain, _ = c.run(share=False)
    assert torch.equal(out[[3, 4]], want[[3, 4]])
    assert torch.equal(out[[0, 2]], plain[[0, 2]]), keep


def test_refusals():
    s = Serve(4, 8, 4, 16)
    q, n = ints([0, 1, 2]), ints([9, 9])
    s.plan(q, n, group_start=ints([0, 2]), prefix_len=ints([5]))
    s.plan(q, n, group_start=ints([0]), prefix_len=ints([])[:0])
    for kw in (dict(group_start=ints([0, 2])), dict(prefix_len=ints([5])), dict(group_start=ints([0, 2]), prefix_len=ints([5, 5])),
               dict(group_start=ints([0, 2]).long(), prefix_len=ints([5])), dict(group_start=ints([0, 2]), prefix_len=ints([5]).cpu())):
        with pytest.raises((TypeError, ValueError)):
            s.plan(q, n, **kw)
    with pytest.raises(B.ColiError) as e:
        s.plan(q, n, group_start=ints([0, 0, 0, 2]), prefix_len=ints([5, 5, 5]))   # more groups than sequences
    assert e.value.status == B.E_INVALID
    s.close()
