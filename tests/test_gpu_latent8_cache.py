"""Rows of an 8-bit latent cache (Serve.append, Serve.read, Serve.keep) against the 64-bit forms: rounding and scales
at ordinary, zero, tiny, huge and infinite values, every byte under every scale, ragged reads of both kinds of
cache, rows that no sequence covers, strides, streams, a captured step, flags and refusals."""
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
from test_gpu_latent_cache import DEV, Kept, Rows, close  # noqa: E402

TYPE = R8.TYPE


def ints(a, kind=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(a)).to(DEV, kind)


def append(s, r, cache, q=True, **kw):
    return s.append(r.c.to(DEV), r.w.to(DEV), 1e-5, r.cos.to(DEV), r.sin.to(DEV), r.pos.to(DEV), r.slots.to(DEV), cache, q_pe=r.q.to(DEV) if q else None, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("n,heads,page", [(1, 1, 1), (7, 5, 16), (130, 64, 64), (33, 3, 2)])
def test_append(n, heads, page, interleaved, dtype):
    r = Rows(n, heads, page, dtype, seed=n)
    cache = torch.full((r.pages, page, R8.ROW8), 0xA5, dtype=torch.uint8, device=DEV)
    s = Serve(heads, n, 1, page, dtype=dtype)
    q = append(s, r, cache, interleaved=interleaved)
    rows, turned = r.want(interleaved)
    flat = cache.view(-1, R8.ROW8).cpu()
    got = flat[r.slots]
    R8.check_rows(got, rows[:, :R.LATENT], dtype)
    close(torch.from_numpy(R8.unpack(got, dtype)[:, R.LATENT:]), rows[:, R.LATENT:], dtype, np.abs(rows).max())
    close(q, turned, dtype, np.abs(turned).max())
    rest = torch.ones(len(flat), dtype=torch.bool)
    rest[r.slots] = False
    assert torch.all(flat[rest] == 0xA5)
    # the same rotary bits and queries as with a 16-bit cache
    other = torch.zeros(r.pages, page, R.ROW, dtype=TYPE[dtype], device=DEV)
    assert torch.equal(append(s, r, other, interleaved=interleaved), q)
    assert torch.equal(other.view(-1, R.ROW).cpu()[r.slots][:, R.LATENT:], got[:, R.LATENT:R.LATENT + 2 * R.ROPE].contiguous().view(TYPE[dtype]))
    assert s.device_errors() == 0
    s.close()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_append_of_extreme_values(dtype):
    """The norm's weights bring the groups to every kind of range: nothing, the least scales, the greatest, beyond the type."""
    r = Rows(3, 1, 16, dtype, seed=5)
    w = torch.ones(R.LATENT)
    big = 2.0 ** 15 if dtype == "f16" else 2.0 ** 124
    for g, by in enumerate([0.0, 2.0 ** -14, 2.0 ** -20, 2.0 ** -9, 1.0, 300.0, big / 16, big / 2, big]):
        w[32 * g:32 * g + 32] = by
    w[32 * 9] = 0.0
    r.w = w.to(TYPE[dtype])
    r.c[0, 64:96] = 0
    r.c[1, ::2] *= 2.0 ** -7
    cache = torch.zeros(r.pages, 16, R8.ROW8, dtype=torch.uint8, device=DEV)
    s = Serve(1, 3, 1, 16, dtype=dtype)
    append(s, r, cache)
    rows, _ = r.want(True)
    R8.check_rows(cache.view(-1, R8.ROW8).cpu()[r.slots], rows[:, :R.LATENT], dtype)
    back = s.read(cache, ints(np.arange(r.pages)[None]), ints([0, r.pages * 16]), n_rows=r.pages * 16)
    assert np.array_equal(back.double().cpu().numpy(), R8.unpack(cache.view(-1, R8.ROW8), dtype), equal_nan=True)
    s.close()


def test_append_of_zeros_and_of_infinities():
    r = Rows(3, 1, 16, "bf16", seed=5)
    r.c[0] = 0
    r.c[1, 7] = float("inf")
    cache = torch.zeros(r.pages, 16, R8.ROW8, dtype=torch.uint8, device=DEV)
    s = Serve(1, 3, 1, 16)
    append(s, r, cache)
    got = R8.unpack(cache.view(-1, R8.ROW8).cpu()[r.slots], "bf16")
    assert np.all(got[0] == 0)
    assert np.isnan(got[1, :R.LATENT]).any()
    r.c[1, 7] = 0
    rows, _ = r.want(True)
    R8.check_rows(cache.view(-1, R8.ROW8).cpu()[r.slots][2:], rows[2:, :R.LATENT], "bf16")
    s.close()


def test_append_without_slots_and_into_one_layer_of_an_interleaved_cache():
    r = Rows(40, 6, 16, "bf16", seed=3)
    s = Serve(6, 40, 1, 16)
    cache = torch.zeros(r.pages, 16, R8.ROW8, dtype=torch.uint8, device=DEV)
    want = append(s, r, cache)
    slots = r.slots.clone()
    r.slots[::3] = -1
    other = torch.full((r.pages, 2, 16, R8.ROW8), 9, dtype=torch.uint8, device=DEV)
    assert torch.equal(append(s, r, other[:, 1]), want)
    assert torch.all(other[:, 0] == 9)
    rows, kept = other[:, 1].reshape(-1, R8.ROW8), r.slots[r.slots >= 0].to(DEV)
    assert torch.equal(rows[kept], cache.view(-1, R8.ROW8)[kept])
    assert torch.all(rows[slots[::3].to(DEV)] == 9)
    r.slots = slots.clone()
    r.slots[1] = r.pages * 16
    append(s, r, cache)
    assert s.device_errors() == 2
    r.slots, r.pos = slots, r.pos.clone()
    r.pos[2] = 500
    append(s, r, cache, q=False)
    assert s.device_errors() == 2
    s.close()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_byte_under_every_scale_reads_back_exactly(dtype):
    """A row per scale and half of the bytes; scales up to the greatest whose 448 (bf16: or 240 at 2^120) is of the type."""
    low, high = R8.LEAST[dtype], R8.MOST[dtype]
    ks = np.arange(low, high + 1)
    rows = np.zeros((len(ks), R8.ROW8), np.uint8)
    rows[:, :512] = np.tile(np.arange(256), 2)
    rows[:, 640:] = (ks + 127)[:, None]
    rows[ks == high, :512][:, 0] = 0
    for b in (0x78, 0x79, 0x7a, 0x7b, 0x7c, 0x7d, 0x7e):          # over 240 at the greatest scale: such rows are not written
        rows[-1][rows[-1] == b] = 0
        rows[-1][:512][rows[-1][:512] == b + 128] = 0
    rows[-1, 640:] = high + 127
    n = len(ks)
    pages = -(-n // 16)
    cache = torch.zeros(pages * 16, R8.ROW8, dtype=torch.uint8)
    cache[:n] = torch.from_numpy(rows)
    s = Serve(1, 1, 1, 16, dtype=dtype)
    out = s.read(cache.view(pages, 16, -1).to(DEV), ints(np.arange(pages)[None]), ints([0, n]), n_rows=n)
    assert np.array_equal(out.double().cpu().numpy(), R8.unpack(cache[:n], dtype), equal_nan=True)
    assert s.device_errors() == 0
    s.close()


class Paged:
    """Sequences of random rows in a cache of either kind, with a first position each."""

    def __init__(self, lens, page, dtype, bits, seed, first=None):
        print(f"read lens={lens[:8]} page={page} {dtype} bits={bits}", flush=True)
        g = torch.Generator().manual_seed(seed)
        self.first = [0] * len(lens) if first is None else first
        each = [-(-(n + f) // page) for n, f in zip(lens, self.first)]
        order = torch.randperm(sum(each) + 1, generator=g)
        self.table = torch.full((len(lens), max(max(each), 1)), -1, dtype=torch.int32)
        at = 0
        for b, e in enumerate(each):
            self.table[b, :e] = order[at:at + e]
            at += e
        latent, rope = torch.randn(len(order), page, R.LATENT, generator=g), torch.randn(len(order), page, R.ROPE, generator=g).to(TYPE[dtype])
        self.cache = torch.cat([latent.to(TYPE[dtype]), rope], -1) if bits == 16 else R8.pack(latent.double().numpy(), rope, dtype)
        self.values = self.cache if bits == 16 else torch.from_numpy(R8.unpack(self.cache, dtype)).to(TYPE[dtype])
        self.lens, self.page = lens, page
        self.k_start = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)

    def want(self):
        rows = []
        for b, n in enumerate(self.lens):
            for i in range(self.first[b], self.first[b] + n):
                rows.append(self.values[self.table[b, i // self.page], i % self.page])
        return torch.stack(rows) if rows else self.values.new_zeros(0, R.ROW)

    def run(self, s, n=None, **kw):
        out = s.read(self.cache.to(DEV), self.table.to(DEV), self.k_start.to(DEV), n_rows=n, first=ints(self.first), **kw)
        torch.cuda.synchronize()
        return out


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("lens,page,first", [([1], 1, None), ([17, 0, 0, 33, 1, 100], 16, None), ([15, 16, 17, 48], 4, [3, 0, 7, 61]), ([0, 0, 5], 64, [200, 1, 0]),
                                             ([3] * 70 + [0] * 130 + [2] * 9, 2, None), ([1000], 64, [23])])
def test_read(lens, page, first, bits, dtype):
    p = Paged(lens, page, dtype, bits, seed=len(lens), first=first)
    s = Serve(1, 1, len(lens), page, dtype=dtype)
    assert torch.equal(p.run(s).cpu(), p.want())
    assert torch.equal(s.read(p.cache.to(DEV), p.table.to(DEV), p.k_start.to(DEV)).cpu()[:0], p.want()[:0])
    assert s.device_errors() == 0 or first is not None
    s.close()


@pytest.mark.parametrize("bits", [8, 16])
def test_read_of_more_sequences_than_a_round_of_the_search(bits):
    r = np.random.default_rng(4)
    p = Paged([int(x) for x in r.integers(0, 4, 5000)], 4, "bf16", bits, seed=2)
    s = Serve(1, 1, 5000, 4)
    assert torch.equal(p.run(s).cpu(), p.want())
    assert s.device_errors() == 0
    s.close()


@pytest.mark.parametrize("bits", [8, 16])
def test_rows_that_no_sequence_covers_and_strides(bits):
    p = Paged([20, 7], 16, "bf16", bits, seed=8)
    s = Serve(1, 1, 2, 16)
    want = p.want()
    wide = torch.full((60, 3, R.ROW + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    out = wide[:, 1, :R.ROW]
    p.k_start = p.k_start + 5                                # rows 5 .. 31
    got = p.run(s, out=out)
    assert got is out and torch.equal(out[5:32].cpu(), want)
    assert torch.all(out[:5] == 7.0) and torch.all(out[32:] == 7.0)
    assert torch.all(wide[:, 0] == 7.0) and torch.all(wide[:, 2] == 7.0) and torch.all(wide[:, 1, R.ROW:] == 7.0)
    assert s.device_errors() == 0
    s.close()


@pytest.mark.parametrize("bits", [8, 16])
def test_read_flags_and_leaves(bits):
    p = Paged([20, 30], 16, "bf16", bits, seed=9)
    s = Serve(1, 1, 2, 16)
    want = p.want()
    for at, value in ((1, -1), (1, len(p.cache)), (0, 1 << 30)):
        bad = Paged([20, 30], 16, "bf16", bits, seed=9)
        bad.table[0, at] = value
        out = torch.full((50, R.ROW), 3.0, dtype=torch.bfloat16, device=DEV)
        bad.run(s, out=out)
        assert s.device_errors() == 2
        assert torch.equal(out[20:].cpu(), want[20:])
    short = Paged([20, 30], 16, "bf16", bits, seed=9)
    short.table = short.table[:, :1].contiguous()
    short.run(s, n=50)
    assert s.device_errors() == 2
    for starts in ([0, 30, 20], [0, 20, 51], [-1, 20, 50]):
        bad = Paged([20, 30], 16, "bf16", bits, seed=9)
        bad.k_start = torch.tensor(starts, dtype=torch.int32)
        bad.run(s, n=50)
        assert s.device_errors() == 1, starts
    bad = Paged([20, 30], 16, "bf16", bits, seed=9)
    bad.first = [-1, 0]
    bad.run(s, n=50)
    assert s.device_errors() == 2
    s.close()


@pytest.mark.parametrize("layers,page", [(1, 16), (3, 4), (2, 64)])
def test_keep(layers, page):
    k = Kept([40, 9, 100, 33, 70], [9, 9, 30, 1, 64], layers, page, seed=layers)
    k.cache = torch.randint(0, 256, (*k.cache.shape[:-1], R8.ROW8), dtype=torch.uint8, generator=torch.Generator().manual_seed(1))
    paths = [[0, 2, 3, 8], [0, 1, 2], [0, 5, 9, 10, 11, 12, 13, 14, 15, 16, 20, 29], [0], list(range(0, 64, 2))]
    s = Serve(1, 113, 5, page)
    assert torch.equal(k.run(s, paths), k.want(paths))
    assert s.device_errors() == 0
    s.close()


def test_append_and_read_captured_and_on_another_stream():
    r = Rows(21, 4, 16, "f16", seed=6)
    s = Serve(4, 21, 1, 16, dtype="f16")
    cache = torch.zeros(r.pages, 16, R8.ROW8, dtype=torch.uint8, device=DEV)
    args = [r.c.to(DEV), r.w.to(DEV), 1e-5, r.cos.to(DEV), r.sin.to(DEV), r.pos.to(DEV), r.slots.to(DEV), cache]
    table, starts, n = ints(np.arange(r.pages)[None]), ints([0, r.pages * 16]), r.pages * 16
    s.append(*args)
    want = s.read(cache, table, starts, n_rows=n)
    side, out = torch.cuda.Stream(), torch.zeros_like(want)
    cache.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.append(*args)
        s.read(cache, table, starts, out=out)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.append(*args)
        s.read(cache, table, starts, out=out)
    for by in (1.0, 2.0, 1.0):
        args[0].copy_(r.c.to(DEV) * by)
        cache.zero_()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        if by == 1.0:
            assert torch.equal(out, want)
        else:
            eager = torch.zeros_like(cache)
            s.append(*args[:-1], eager)
            assert torch.equal(out, s.read(eager, table, starts, n_rows=n))
    s.close()


def test_refusals():
    p = Paged([20, 30], 16, "bf16", 8, seed=9)
    s = Serve(2, 1, 2, 16)
    good = dict(cache=p.cache.to(DEV), block_table=p.table.to(DEV), k_start=p.k_start.to(DEV), n_rows=50)
    s.read(**good)
    for name, bad in (("cache", good["cache"].to(torch.int8)), ("cache", good["cache"][..., :640]), ("cache", good["cache"][:, :8]), ("cache", good["cache"].cpu()), ("block_table", p.table.long().to(DEV)),
                      ("k_start", good["k_start"].long()), ("k_start", good["k_start"][:2]), ("first", ints([0])), ("n_rows", -1), ("out", torch.zeros(50, R.ROW, device=DEV)),
                      ("out", torch.zeros(49, R.ROW, device=DEV).bfloat16())):
        with pytest.raises((TypeError, ValueError)):
            s.read(**{**good, name: bad})
    odd = torch.zeros(50 * R.ROW + 1, dtype=torch.bfloat16, device=DEV)[1:].view(50, R.ROW)
    with pytest.raises(B.ColiError) as e:
        s.read(**good, out=odd)
    assert e.value.status == B.E_INVALID
    shifted = torch.zeros(good["cache"].numel() + 8, dtype=torch.uint8, device=DEV)[8:].view(good["cache"].shape)
    with pytest.raises(B.ColiError) as e:
        s.read(**{**good, "cache": shifted})
    assert e.value.status == B.E_INVALID and "aligned" in str(e.value)
    assert s.read(good["cache"], good["block_table"], ints([0, 0, 0]), n_rows=0).shape == (0, R.ROW)
    s.close()
