"""Rows of the latent cache (Serve.append, Serve.keep) against the 64-bit forms:
both rotary orders, pages of one row and more, tokens without a slot, strides,
in-place queries, flags; kept rows over layers, overlapping moves, long paths."""
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


class Rows:
    def __init__(self, n, heads, page, dtype, seed):
        print(f"append n={n} heads={heads} page={page} {dtype} seed={seed}", flush=True)
        g = torch.Generator().manual_seed(seed)
        dt = TYPE[dtype]
        self.pages = -(-n // page) + 2
        self.c = (3 * torch.randn(n, R.ROW, generator=g)).to(dt)
        self.w = (1 + 0.2 * torch.randn(R.LATENT, generator=g)).to(dt)
        angle = torch.arange(500)[:, None] * 10000.0 ** (-torch.arange(32) / 32)
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        self.pos = torch.randint(0, 500, (n,), generator=g).int()
        self.slots = torch.randperm(self.pages * page, generator=g)[:n]
        self.q = torch.randn(n, heads, R.ROPE, generator=g).to(dt)

    def want(self, interleaved):
        cos, sin = self.cos[self.pos.long()].double().numpy(), self.sin[self.pos.long()].double().numpy()
        rows = R.norm_rows(self.c.double().numpy(), self.w.double().numpy(), 1e-5, cos, sin, interleaved)
        return rows, R.rotate(self.q.double().numpy(), cos[:, None], sin[:, None], interleaved)


def close(got, want, dtype, size):
    """One rounding, on values computed in fp32 to a few units of their terms."""
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= R.UNIT[dtype] * np.abs(want) + 2.0 ** -20 * size + 2.0 ** -25)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("n,heads,page", [(1, 1, 1), (7, 5, 16), (130, 64, 64), (33, 3, 2)])
def test_append(n, heads, page, interleaved, dtype):
    r = Rows(n, heads, page, dtype, seed=n)
    cache = torch.full((r.pages, page, R.ROW), 5.0, dtype=TYPE[dtype], device=DEV)
    s = Serve(heads, n, 1, page, dtype=dtype)
    q = s.append(r.c.to(DEV), r.w.to(DEV), 1e-5, r.cos.to(DEV), r.sin.to(DEV), r.pos.to(DEV), r.slots.to(DEV), cache, q_pe=r.q.to(DEV), interleaved=interleaved)
    rows, turned = r.want(interleaved)
    flat = cache.view(-1, R.ROW).cpu()
    close(flat[r.slots], rows, dtype, np.abs(rows).max())
    close(q, turned, dtype, np.abs(turned).max())
    rest = torch.ones(len(flat), dtype=torch.bool)
    rest[r.slots] = False
    assert torch.all(flat[rest] == 5.0)
    assert s.device_errors() == 0
    s.close()


def test_append_without_slots_in_place_and_strided():
    r = Rows(40, 6, 16, "bf16", seed=3)
    s = Serve(6, 40, 1, 16)
    cache = torch.zeros(r.pages, 16, R.ROW, dtype=torch.bfloat16, device=DEV)
    args = (r.w.to(DEV), 1e-5, r.cos.to(DEV), r.sin.to(DEV), r.pos.to(DEV))
    want = s.append(r.c.to(DEV), *args, r.slots.to(DEV), cache, q_pe=r.q.to(DEV))
    slots = r.slots.clone()
    slots[::3] = -1
    wide = torch.full((40, 2, R.ROW + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 1, 8:8 + R.ROW] = r.c.to(DEV)
    q = r.q.to(DEV)
    other = torch.full((r.pages, 2, 16, R.ROW), 9.0, dtype=torch.bfloat16, device=DEV)
    got = s.append(wide[:, 1, 8:8 + R.ROW], *args, slots.to(DEV), other[:, 1], q_pe=q, q_out=q)
    assert got is q and torch.equal(q, want)
    assert torch.all(other[:, 0] == 9.0)
    rows = other[:, 1].reshape(-1, R.ROW)
    kept = slots[slots >= 0].to(DEV)
    assert torch.equal(rows[kept], cache.view(-1, R.ROW)[kept])
    assert torch.all(rows[r.slots[::3].to(DEV)] == 9.0)
    assert s.append(r.c.to(DEV), *args, r.slots.to(DEV), cache) is None
    assert s.device_errors() == 0
    s.close()


def test_append_flags_slots_and_positions_out_of_range():
    r = Rows(4, 2, 16, "bf16", seed=4)
    s = Serve(2, 4, 1, 16)
    cache = torch.zeros(r.pages, 16, R.ROW, dtype=torch.bfloat16, device=DEV)
    call = lambda pos, slots: s.append(r.c.to(DEV), r.w.to(DEV), 1e-5, r.cos.to(DEV), r.sin.to(DEV), pos.to(DEV), slots.to(DEV), cache, q_pe=r.q.to(DEV))  # noqa: E731
    for slot in (r.pages * 16, 1 << 40):
        slots = r.slots.clone()
        slots[1] = slot
        call(r.pos, slots)
        assert s.device_errors() == 2
    for pos in (-1, 500):
        bad = r.pos.clone()
        bad[2] = pos
        call(bad, r.slots)
        assert s.device_errors() == 2
    s.close()


def test_append_of_zeros_and_of_infinities():
    """A row of zeros stays zeros; a row that is not finite spoils only itself."""
    r = Rows(3, 1, 16, "bf16", seed=5)
    r.c[0] = 0
    r.c[1, 7] = float("inf")
    cache = torch.zeros(r.pages, 16, R.ROW, dtype=torch.bfloat16, device=DEV)
    s = Serve(1, 3, 1, 16)
    s.append(r.c.to(DEV), r.w.to(DEV), 1e-5, r.cos.to(DEV), r.sin.to(DEV), r.pos.to(DEV), r.slots.to(DEV), cache)
    flat = cache.view(-1, R.ROW)[r.slots.to(DEV)]
    assert torch.all(flat[0] == 0)
    assert not torch.isfinite(flat[1, :R.LATENT]).all()
    r.c[1, 7] = 0
    rows, _ = r.want(True)
    close(flat[2], rows[2], "bf16", np.abs(rows[2]).max())
    s.close()


class Kept:
    def __init__(self, lens, nodes, layers, page, seed, spare=1):
        print(f"keep lens={lens} nodes={nodes} layers={layers} page={page}", flush=True)
        g = torch.Generator().manual_seed(seed)
        each = [-(-n // page) for n in lens]
        order = torch.randperm(sum(each) + spare, generator=g).int()
        self.table = torch.full((len(lens), max(each)), -1, dtype=torch.int32)
        at = 0
        for b, e in enumerate(each):
            self.table[b, :e] = order[at:at + e]
            at += e
        self.cache = torch.randn(layers, len(order), page, R.ROW, generator=g).bfloat16()
        self.lens, self.nodes, self.page = lens, nodes, page
        self.q_start = torch.tensor(np.concatenate([[0], np.cumsum(nodes)]), dtype=torch.int32)

    def want(self, paths):
        out = self.cache.clone()
        for b, path in enumerate(paths):
            base = self.lens[b] - self.nodes[b]
            for i, n in enumerate(path):
                to, at = base + i, base + n
                out[:, self.table[b, to // self.page], to % self.page] = self.cache[:, self.table[b, at // self.page], at % self.page]
        return out

    def run(self, serve, paths, cols=None):
        cols = cols or max(len(p) for p in paths)
        t = torch.full((len(paths), cols), -1, dtype=torch.int32)
        for b, p in enumerate(paths):
            t[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        cache = self.cache.to(DEV)
        serve.keep(cache, self.table.to(DEV), self.q_start.to(DEV), torch.tensor(self.lens, dtype=torch.int32, device=DEV), t.to(DEV))
        torch.cuda.synchronize()
        return cache.cpu()


@pytest.mark.parametrize("layers,page", [(1, 16), (3, 4), (2, 64)])
def test_keep(layers, page):
    k = Kept([40, 9, 100, 33, 70], [9, 9, 30, 1, 64], layers, page, seed=layers)
    paths = [[0, 2, 3, 8], [0, 1, 2], [0, 5, 9, 10, 11, 12, 13, 14, 15, 16, 20, 29], [0], list(range(0, 64, 2))]
    s = Serve(1, 113, 5, page)
    assert torch.equal(k.run(s, paths), k.want(paths))
    assert s.device_errors() == 0
    one = Kept([40], [9], 1, page, seed=9)                  # a cache of one layer without the leading dimension
    cache = one.cache[0].to(DEV)
    s.keep(cache, one.table.to(DEV), one.q_start.to(DEV), torch.tensor([40], dtype=torch.int32, device=DEV), torch.tensor([[0, 3, 7]], dtype=torch.int32, device=DEV))
    assert torch.equal(cache.cpu(), one.want([[0, 3, 7]])[0])
    s.close()


def test_keep_of_nothing_and_flags():
    k = Kept([20, 30], [5, 4], 1, 16, seed=7)
    s = Serve(1, 9, 2, 16)
    same = k.run(s, [[], []], cols=3)
    assert torch.equal(same, k.cache) and s.device_errors() == 0
    for path in ([0, 5], [0, 2, 1], [1, 0]):                # past the nodes, descending: stops there
        k.run(s, [path, [0]])
        assert s.device_errors() == 4, path
    k.table[1, 1] = 99
    k.run(s, [[0], [0, 3]])
    assert s.device_errors() == 2
    k.lens = [4, 30]                                        # more nodes than cached positions
    k.run(s, [[0, 2], [0]])
    assert s.device_errors() == 1
    s.close()


def test_refusals():
    s = Serve(2, 8, 2, 16)
    r = Rows(4, 2, 16, "bf16", seed=6)
    cache = torch.zeros(r.pages, 16, R.ROW, dtype=torch.bfloat16, device=DEV)
    good = dict(c=r.c.to(DEV), norm_weight=r.w.to(DEV), eps=1e-5, cos=r.cos.to(DEV), sin=r.sin.to(DEV), positions=r.pos.to(DEV), slots=r.slots.to(DEV), cache=cache)
    s.append(**good)
    for name, bad in (("c", good["c"].float()), ("c", good["c"][:, :512]), ("norm_weight", good["norm_weight"][:5]), ("cos", good["cos"].double()), ("sin", good["sin"][:9]),
                      ("positions", good["positions"].long()), ("slots", good["slots"].int()), ("cache", cache[:, :4]), ("cache", cache.cpu()), ("slots", None)):
        with pytest.raises((TypeError, ValueError)):
            s.append(**{**good, name: bad})
    with pytest.raises(ValueError):
        s.append(**good, q_out=r.q.to(DEV))
    with pytest.raises(B.ColiError) as e:
        s.append(**{**good, "eps": float("nan")})
    assert e.value.status == B.E_INVALID
    odd = torch.zeros(4 * 580, dtype=torch.bfloat16, device=DEV).view(4, 580)[:, 3:579]
    with pytest.raises(B.ColiError) as e:
        s.append(**{**good, "c": odd})
    assert e.value.status == B.E_INVALID
    k = Kept([20], [5], 1, 16, seed=8)
    args = [k.cache.to(DEV), k.table.to(DEV), k.q_start.to(DEV), torch.tensor([20], dtype=torch.int32, device=DEV), torch.tensor([[0]], dtype=torch.int32, device=DEV)]
    s.keep(*args)
    for i, bad in ((0, args[0].half()), (1, args[1].long()), (2, args[2][:0]), (3, args[3].repeat(2)), (4, args[4][0])):
        with pytest.raises((TypeError, ValueError)):
            s.keep(*[bad if j == i else a for j, a in enumerate(args)])
    s.close()
