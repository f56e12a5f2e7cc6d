"""Beam selection (Serve.beam_select) and reordering (Serve.beam_reorder) against their 64-bit and plain forms: types,
odd vocabularies, strides, beams that are dead, ties within and between beams, rows without or with infinite logits, more kept
than there are; every exchange of beams, forks, pages that are full, layers, both kinds of cache; streams, graphs, flags, refusals."""
import itertools

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

DEV = "cuda:0"
TYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def ints(a):
    return torch.as_tensor(np.ascontiguousarray(a)).to(DEV, torch.int32)


def check(s, logits, scores, keep, flags=0):
    """logits [g, b, v] on the host, scores [g, b].  Scores are off by the rounding to fp32 and by the logarithm of a sum of
    fp32 exponentials: of each the exponent is off by 2^-24 of itself (24 at most where it counts), the exponential by two
    units more, and a thread's sum of 32 terms by 32: 2^-24 (24 + 2 + 32 + 8)."""
    g, b, v = logits.shape
    print(f"select {g}x{b}x{v} keep={keep} {logits.dtype}", flush=True)
    want = R8.select(logits.double().numpy(), scores.double().numpy(), keep)
    got = s.beam_select(logits.view(g * b, v).to(DEV), scores.to(DEV), keep)
    assert s.device_errors() == flags
    best, parents, tokens = (x.cpu().numpy() for x in got)
    assert np.array_equal(parents, want[1]) and np.array_equal(tokens, want[2])
    live = parents >= 0
    assert np.all(np.isneginf(best[~live]))
    assert np.all(np.abs(best[live] - want[0][live]) <= 2.0 ** -24 * (66 + np.abs(want[0][live])))
    return got


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("g,b,v,keep", [(1, 1, 1, 1), (2, 3, 2, 5), (1, 4, 2047, 8), (3, 2, 2048, 4), (2, 5, 2049, 64), (1, 64, 300, 64), (7, 8, 8193, 16), (1, 2, 100003, 40), (40, 16, 8192, 3)])
def test_select(g, b, v, keep, kind):
    r = torch.Generator().manual_seed(v + keep)
    logits = (3 * torch.randn(g, b, v, generator=r)).to(TYPE[kind])
    scores = -4 * torch.rand(g, b, generator=r)
    s = Serve(1, 1, g * b)
    check(s, logits, scores, keep)
    s.close()


def test_large_chunks_of_a_large_batch():
    r = torch.Generator().manual_seed(1)
    s = Serve(1, 1, 64)
    check(s, 2 * torch.randn(8, 8, 151643, generator=r), -torch.rand(8, 8, generator=r), 17)
    s.close()


@pytest.mark.parametrize("v", [50, 5000, 40000])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_ties(v, kind):
    """Equal logits, few values, equal beams: the lower beam first, then the lower token."""
    s = Serve(1, 1, 256)
    check(s, torch.zeros(2, 4, v).to(TYPE[kind]), torch.zeros(2, 4), 20)
    r = torch.Generator().manual_seed(2)
    check(s, torch.randint(-2, 3, (2, 4, v), generator=r).to(TYPE[kind]), torch.full((2, 4), -1.5), 64)
    same = (3 * torch.randn(1, 1, v, generator=r)).to(TYPE[kind]).expand(2, 64, v).contiguous()
    check(s, same, torch.full((2, 64), -2.0), 33)
    check(s, torch.zeros(1, 64, v).to(TYPE[kind]), torch.zeros(1, 64), 64)
    zeros = torch.zeros(1, 2, v)
    zeros[0, :, 1::2] = -0.0
    check(s, zeros.to(TYPE[kind]), torch.zeros(1, 2), 9)
    s.close()


def test_values_in_falling_order_along_a_thread():
    """All large values lie where one thread loads them, in four neighbours at a time."""
    x = torch.arange(16384, 0, -1).float().view(1, 1, -1) / 512
    s = Serve(1, 1, 1)
    check(s, x, torch.zeros(1, 1), 64)
    check(s, x.flip(2).contiguous(), torch.zeros(1, 1), 64)
    y = torch.full((1, 1, 16384), -5.0)
    y[0, 0, :128] = torch.linspace(1, 9, 128)
    check(s, y, torch.zeros(1, 1), 64)
    s.close()


def test_dead_beams_masked_tokens_and_fewer_than_kept():
    r = torch.Generator().manual_seed(3)
    logits = torch.randn(4, 3, 70, generator=r)
    scores = -torch.rand(4, 3, generator=r)
    scores[0, 1:] = -float("inf")                            # the first step of a search: one beam lives
    scores[1] = -float("inf")                                # none
    scores[2, 0], scores[2, 1] = float("nan"), float("inf")
    logits[3, :, 2:] = -float("inf")                         # a constraint that leaves two tokens
    logits[3, 1, 0] = float("nan")
    s = Serve(1, 1, 12)
    check(s, logits, scores, 8)
    s.close()


def test_rows_of_no_value_set_a_flag():
    r = torch.Generator().manual_seed(4)
    s = Serve(1, 1, 4)
    for value in (-float("inf"), float("nan")):
        logits = torch.randn(2, 2, 5000, generator=r)
        logits[0, 1] = value
        check(s, logits, torch.zeros(2, 2), 6, flags=8)
        dead = torch.tensor([[0.0, -float("inf")], [0.0, 0.0]])
        check(s, logits, dead, 6)                            # of a dead beam: nobody looks
    logits = torch.randn(2, 2, 5000, generator=r)
    logits[1, 0, 77] = float("inf")
    check(s, logits, torch.zeros(2, 2), 6, flags=8)
    s.close()


def test_scores_beyond_the_range_of_fp32_differences():
    s = Serve(1, 1, 2)
    logits = torch.zeros(1, 2, 3000)
    logits[0, 0, 5], logits[0, 0, 6] = 3e38, -3e38
    logits[0, 1, 7] = -3e38
    check(s, logits, torch.tensor([[0.0, -3e38]]), 4)
    s.close()


@pytest.mark.parametrize("kind", ["f32", "f16"])
def test_strided_rows_and_odd_addresses(kind):
    r = torch.Generator().manual_seed(5)
    logits = torch.randn(2, 3, 1001, generator=r).to(TYPE[kind])
    s = Serve(1, 1, 6)
    want = check(s, logits, torch.zeros(2, 3), 7)
    wide = torch.full((6, 1100), float("nan"), dtype=TYPE[kind], device=DEV)
    wide[:, 13:1014] = logits.view(6, -1).to(DEV)
    got = s.beam_select(wide[:, 13:1014], torch.zeros(2, 3, device=DEV), 7)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    s.close()


def test_select_captured_and_on_another_stream():
    r = torch.Generator().manual_seed(6)
    s = Serve(1, 1, 8)
    a, b = (3 * torch.randn(8, 30011, generator=r).to(DEV) for _ in range(2))
    scores = -torch.rand(2, 4, generator=r).to(DEV)
    want = {k: [x.clone() for x in s.beam_select(x, scores, 8)] for k, x in (("a", a), ("b", b))}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = s.beam_select(a, scores, 8)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want["a"]))
    logits = a.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = s.beam_select(logits, scores, 8)
    for k, x in (("b", b), ("a", a), ("b", b)):
        logits.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want[k]))
        s.beam_select(a, scores, 64)                         # the same scratch, between replays
    s.close()


def test_select_refusals():
    s = Serve(1, 1, 6)
    logits, scores = torch.zeros(6, 100, device=DEV), torch.zeros(2, 3, device=DEV)
    s.beam_select(logits, scores, 4)
    for a in ((logits.double(), scores, 4), (logits.cpu(), scores, 4), (logits, scores.half(), 4), (logits[:5], scores, 4), (logits, scores[0], 4), (logits.t().contiguous().t(), scores, 4),
              (logits, scores, 0)):
        with pytest.raises((TypeError, ValueError)):
            s.beam_select(*a)
    for a in ((logits, scores, 65), (torch.zeros(12, 100, device=DEV), torch.zeros(4, 3, device=DEV), 4), (logits[:, :0], scores, 1)):
        with pytest.raises(B.ColiError) as e:
            s.beam_select(*a)
        assert e.value.status == B.E_INVALID
    with pytest.raises(B.ColiError) as e:
        s.beam_select(torch.zeros(6, (1 << 20) + 1, dtype=torch.bfloat16, device=DEV), scores, 4)
    assert e.value.status == B.E_UNSUPPORTED
    assert [tuple(x.shape) for x in s.beam_select(logits[:0], scores[:0], 4)] == [(0, 4)] * 3
    s.close()


class Beams:
    """Groups of beams of `lens` positions: shared whole pages, own ones from that of the length on."""

    def __init__(self, lens, beams, page, layers, bits, seed, room=1):
        print(f"reorder lens={lens[:6]} beams={beams} page={page} layers={layers} bits={bits}", flush=True)
        g = torch.Generator().manual_seed(seed)
        cols = max(lens) // page + room
        tables, n = [], 0
        for ln in lens:
            whole = ln // page
            shared = list(range(n, n + whole))
            n += whole
            for _ in range(beams):
                own = list(range(n, n + cols - whole))
                n += cols - whole
                tables.append(shared + own)
        order = torch.randperm(n + 1, generator=g)
        self.table = order[torch.tensor(tables).long()].int().view(len(tables), cols)
        shape = (layers, n + 1, page)
        self.cache = torch.randint(0, 256, (*shape, R8.ROW8), dtype=torch.uint8, generator=g) if bits == 8 else torch.randn(*shape, R.ROW, generator=g).bfloat16()
        self.lens, self.beams, self.page = lens, beams, page

    def run(self, s, parents, **kw):
        cache = self.cache.to(DEV)
        table = s.beam_reorder(cache, self.table.to(DEV), ints(np.repeat(self.lens, self.beams)), ints(parents), **kw)
        torch.cuda.synchronize()
        return cache.cpu(), table.cpu()

    def check(self, s, parents, flags=0):
        cache, table = self.run(s, parents)
        assert s.device_errors() == flags
        want_cache, want_table = R8.reorder(self.cache, self.table, self.lens, np.asarray(parents), self.page)
        assert torch.equal(table, want_table)
        assert torch.equal(cache.view(torch.uint8), want_cache.view(torch.uint8))
        for i, ln in enumerate(self.lens):                   # from the page of the length on nothing is shared
            own = table[i * self.beams:(i + 1) * self.beams, ln // self.page:].flatten().tolist()
            assert len(set(own)) == len(own)


@pytest.mark.parametrize("bits", [16, 8])
def test_every_exchange_of_three_beams(bits):
    every = list(itertools.product([-1, 0, 1, 2], repeat=3))
    b = Beams([1 + 5 * i % 37 for i in range(len(every))], 3, 8, 1, bits, seed=1)
    s = Serve(1, 1, 3 * len(every), 8)
    b.check(s, every)
    s.close()


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("beams,page,layers", [(1, 16, 1), (2, 1, 3), (8, 16, 2), (64, 4, 1), (5, 64, 4)])
def test_reorder(beams, page, layers, bits):
    r = np.random.default_rng(beams)
    lens = [0, page, 3 * page - 1, page // 2, 2 * page + 1]
    b = Beams(lens, beams, page, layers, bits, seed=beams, room=3)
    s = Serve(1, 1, beams * len(lens), page)
    b.check(s, r.integers(0, beams, (len(lens), beams)))
    b.check(s, np.tile(np.arange(beams), (len(lens), 1)))    # nothing moves
    b.check(s, np.zeros((len(lens), beams), int))            # forks
    b.check(s, np.full((len(lens), beams), beams - 1))
    s.close()


def test_a_table_that_is_full():
    b = Beams([32, 16], 3, 16, 1, 16, seed=7, room=0)
    s = Serve(1, 1, 6, 16)
    b.check(s, [[2, 2, 0], [1, 1, 1]])
    s.close()


def test_a_cache_of_one_layer_and_strided_tables():
    b = Beams([37, 20], 4, 16, 1, 8, seed=8)
    parents = [[1, 1, 3, 1], [0, 2, 2, 0]]
    s = Serve(1, 1, 8, 16)
    want_cache, want_table = R8.reorder(b.cache, b.table, b.lens, np.asarray(parents), 16)
    cols = b.table.shape[1]
    wide = torch.full((8, cols + 5), -1, dtype=torch.int32, device=DEV)
    wide[:, 2:2 + cols] = b.table.to(DEV)
    out = torch.full((8, cols + 3), 77, dtype=torch.int32, device=DEV)
    pages = torch.full((b.cache.shape[1], 2, 16, R8.ROW8), 5, dtype=torch.uint8, device=DEV)
    pages[:, 1] = b.cache[0].to(DEV)
    got = s.beam_reorder(pages[:, 1], wide[:, 2:2 + cols], ints(np.repeat(b.lens, 4)), ints(parents), out=out[:, 1:1 + cols])
    assert torch.equal(got.cpu(), want_table) and torch.all(out[:, 0] == 77) and torch.all(out[:, 1 + cols:] == 77)
    assert torch.equal(pages[:, 1].cpu(), want_cache[0]) and torch.all(pages[:, 0] == 5)
    assert s.device_errors() == 0
    s.close()


def test_reorder_flags():
    s = Serve(1, 1, 6, 16)
    for parents in ([[3, 0, 0], [0, 1, 1]], [[-2, 0, 0], [0, 1, 1]], [[1 << 30, 0, 0], [0, 1, 1]]):
        Beams([20, 9], 3, 16, 2, 16, seed=9).check(s, parents, flags=4)
    b = Beams([20, 9], 3, 16, 2, 16, seed=9)
    for lens in ([20, 21, 20, 9, 9, 9], [-1, -1, -1, 9, 9, 9]):
        cache = b.cache.to(DEV)
        table = s.beam_reorder(cache, b.table.to(DEV), ints(lens), ints([[0, 0, 0], [0, 1, 1]])).cpu()
        assert s.device_errors() == 1
        want_cache, want_table = R8.reorder(b.cache, b.table, b.lens, np.array([[0, 1, 2], [0, 1, 1]]), 16)
        assert torch.equal(table, want_table) and torch.equal(cache.cpu(), want_cache)
    for value in (-1, 10 ** 6):
        bad = Beams([20, 9], 3, 16, 2, 16, seed=9)
        bad.table[1, 1] = value                              # beam 1's last page, which place 1 takes over
        cache, table = bad.run(s, [[0, 0, 2], [0, 1, 2]])
        assert s.device_errors() == 2
        assert torch.equal(cache, bad.cache)
    short = Beams([20, 9], 3, 16, 2, 16, seed=9)
    short.table = short.table[:, :1].contiguous()            # no column for the last page of the first group
    cache, _ = short.run(s, [[0, 0, 2], [0, 1, 2]])
    assert s.device_errors() == 2 and torch.equal(cache, short.cache)
    s.close()


def test_reorder_captured_and_on_another_stream():
    b = Beams([37, 20], 4, 16, 2, 8, seed=10)
    s = Serve(1, 1, 8, 16)
    cache, table, lens, parents = b.cache.to(DEV), b.table.to(DEV), ints(np.repeat(b.lens, 4)), ints([[1, 1, 3, 1], [0, 2, 2, 0]])
    out = torch.zeros_like(table)
    want = b.run(s, parents.cpu().numpy())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.beam_reorder(cache, table, lens, parents, out=out)
    side.synchronize()
    assert torch.equal(out.cpu(), want[1]) and torch.equal(cache.cpu(), want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.beam_reorder(cache, table, lens, parents, out=out)
    for p in ([[0, 1, 2, 3]] * 2, [[3, 3, 3, 0], [-1, 1, 1, 1]], [[1, 1, 3, 1], [0, 2, 2, 0]]):
        parents.copy_(ints(p))
        cache.copy_(b.cache.to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        want = b.run(s, p)
        assert torch.equal(out.cpu(), want[1]) and torch.equal(cache.cpu(), want[0])
    s.close()


def test_reorder_refusals():
    b = Beams([20, 9], 3, 16, 1, 16, seed=11)
    s = Serve(1, 1, 6, 16)
    good = dict(cache=b.cache.to(DEV), block_table=b.table.to(DEV), kv_len=ints(np.repeat(b.lens, 3)), parents=ints([[0, 1, 2]] * 2))
    s.beam_reorder(**good)
    for name, bad in (("parents", good["parents"].long()), ("parents", good["parents"][0]), ("parents", good["parents"][:1]), ("kv_len", good["kv_len"][:2]), ("block_table", good["block_table"].cpu()),
                      ("cache", good["cache"].half()), ("out", good["block_table"].long()), ("out", good["block_table"][:, :1])):
        with pytest.raises((TypeError, ValueError)):
            s.beam_reorder(**{**good, name: bad})
    for out in (good["block_table"], ):
        with pytest.raises(B.ColiError) as e:
            s.beam_reorder(**good, out=out)
        assert e.value.status == B.E_INVALID and "overlap" in str(e.value)
    small = Serve(1, 1, 5, 16)
    with pytest.raises(B.ColiError) as e:
        small.beam_reorder(**good)
    assert e.value.status == B.E_INVALID
    many = torch.zeros(1, 65, dtype=torch.int32, device=DEV)
    big = Serve(1, 1, 65, 16)
    with pytest.raises(B.ColiError) as e:
        big.beam_reorder(good["cache"], torch.zeros(65, 1, dtype=torch.int32, device=DEV), many[0].contiguous(), many)
    assert e.value.status == B.E_INVALID
    for x in (s, small, big):
        x.close()
