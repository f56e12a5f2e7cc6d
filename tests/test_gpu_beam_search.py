"""Append, read, shared-prefix attention, selection and reordering together, as a beam search over an 8-bit cache uses them: a toy
decoder whose rows, queries and logits follow from the tokens alone, so that the cache of every beam can be written down from its history."""
import numpy as np
import pytest

import serve8_case as R8
import serve_case as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from int4_routed_expert_layer_amd.serve import Serve  # noqa: E402

DEV = "cuda:0"
VOCAB, HEADS, PAGE, BEAMS, STEPS = 211, 6, 16, 4, 40
U = 2.0 ** -8      # unit roundoff of bf16


class Toy:
    def __init__(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def normal(*shape, by=1.0):
            return (by * torch.randn(shape, generator=g, device=DEV)).bfloat16()

        self.row, self.q_lat, self.q_pe = normal(VOCAB, R.ROW), normal(VOCAB, HEADS, R.LATENT, by=0.2), normal(VOCAB, HEADS, R.ROPE, by=0.2)
        self.norm = (1 + 0.1 * torch.randn(R.LATENT, generator=g, device=DEV)).bfloat16()
        self.head = normal(HEADS * R.LATENT, VOCAB, by=0.15)
        angle = torch.arange(500, device=DEV)[:, None] * 10000.0 ** (-torch.arange(32, device=DEV) / 32)
        self.cos, self.sin = angle.cos().float().contiguous(), angle.sin().float().contiguous()

    def append(self, s, tokens, positions, slots, cache):
        t = tokens.long()
        return s.append(self.row[t], self.norm, 1e-6, self.cos, self.sin, positions, slots, cache, q_pe=self.q_pe[t])


def ints(a, kind=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(a)).to(DEV, kind)


def rows_of(toy, s, tokens, bits):
    """The cache rows of a sequence of tokens at positions 0, 1 ..."""
    n = len(tokens)
    cache = torch.zeros(-(-n // PAGE), PAGE, R8.ROW8, dtype=torch.uint8, device=DEV) if bits == 8 else torch.zeros(-(-n // PAGE), PAGE, R.ROW, dtype=torch.bfloat16, device=DEV)
    toy.append(s, ints(tokens), ints(np.arange(n)), ints(np.arange(n), torch.int64), cache)
    return cache.view(-1, cache.shape[-1])[:n]


@pytest.mark.parametrize("bits", [8, 16])
def test_beam_search(bits):
    toy, r = Toy(1), np.random.default_rng(2)
    prompts = [r.integers(0, VOCAB, n).tolist() for n in (70, 133)]
    groups, n = len(prompts), len(prompts) * BEAMS
    s = Serve(HEADS, n, n, PAGE)
    s_all = Serve(HEADS, 512, n, PAGE)
    cols = (max(map(len, prompts)) + STEPS) // PAGE + 1
    table, used = np.full((n, cols), -1), 0
    for i, p in enumerate(prompts):                          # beam 0 has the prompt's pages, all have own ones from the last on
        whole = len(p) // PAGE
        table[i * BEAMS, :whole] = np.arange(used, used + whole)
        used += whole
        for j in range(BEAMS):
            table[i * BEAMS + j, whole:] = np.arange(used, used + cols - whole)
            used += cols - whole
    cache = torch.full((used, PAGE, R8.ROW8), 0xFF, dtype=torch.uint8, device=DEV) if bits == 8 else torch.full((used, PAGE, R.ROW), float("nan"), dtype=torch.bfloat16, device=DEV)
    # all but a prompt's last token are cached; the last is each beam's first step
    for i, p in enumerate(prompts):
        pos = np.arange(len(p) - 1)
        toy.append(s_all, ints(p[:-1]), ints(pos), ints(table[i * BEAMS, pos // PAGE] * PAGE + pos % PAGE, torch.int64), cache)
    lens = ints(np.repeat([len(p) - 1 for p in prompts], BEAMS))
    table = s.beam_reorder(cache, ints(table), lens, ints(np.zeros((groups, BEAMS), int)))   # fork
    q_start, starts, prefix = ints(np.arange(n + 1)), ints(np.arange(groups + 1) * BEAMS), ints([len(p) - 1 for p in prompts])
    scores = torch.full((groups, BEAMS), -float("inf"), device=DEV)
    scores[:, 0] = 0.0
    tokens = ints(np.repeat([p[-1] for p in prompts], BEAMS))
    history = [list(p) for p in prompts for _ in range(BEAMS)]
    offset = torch.arange(groups, device=DEV)[:, None] * BEAMS
    for step in range(STEPS):
        page = torch.gather(table.long(), 1, (lens.long() // PAGE)[:, None])[:, 0]
        q_pe = toy.append(s, tokens, lens, page * PAGE + lens.long() % PAGE, cache)
        lens = lens + 1
        q_lat = toy.q_lat[tokens.long()]
        s.plan(q_start, lens, n_tok=n, group_start=starts, prefix_len=prefix)
        out = s.decode(q_lat, q_pe, cache, table, 1 / 16)
        if step in (0, 17, STEPS - 1):
            s_all.plan(q_start, lens, n_tok=n)
            apart = s_all.decode(q_lat, q_pe, cache, table, 1 / 16)
            # the same rows in other pieces: weights rounded against other maxima, and the result's rounding, twice
            assert torch.all((out.float() - apart.float()).abs() <= 4 * U * apart.float().abs().amax(-1, keepdim=True))
        logits = (out.flatten(1).float() @ toy.head.float()).contiguous()
        want = R8.select(logits.view(groups, BEAMS, VOCAB).double().cpu().numpy(), scores.double().cpu().numpy(), BEAMS)
        scores, parents, new = s.beam_select(logits, scores, BEAMS)
        assert np.array_equal(parents.cpu().numpy(), want[1]) and np.array_equal(new.cpu().numpy(), want[2])
        table = s.beam_reorder(cache, table, lens, parents)
        tokens = new.flatten()
        scores = scores.contiguous()
        flat = (parents + offset).flatten().tolist()
        history = [history[p] + [t] for p, t in zip(flat, tokens.tolist())]
    assert s.device_errors() == 0 and s_all.device_errors() == 0
    got = s.read(cache, table, ints(np.concatenate([[0], np.cumsum(lens.tolist())])), n_rows=int(lens.sum()))
    at = 0
    for b in range(n):
        rows = rows_of(toy, s_all, history[b][:-1], bits)     # the newest token is not cached yet
        m = len(rows)
        pos = np.arange(m)
        mine = cache.view(-1, cache.shape[-1])[ints(table[b].cpu().numpy()[pos // PAGE] * PAGE + pos % PAGE, torch.int64)]
        assert torch.equal(mine.view(torch.uint8), rows.contiguous().view(torch.uint8)), b
        values = torch.from_numpy(R8.unpack(rows, "bf16")).to(DEV).bfloat16() if bits == 8 else rows
        assert torch.equal(got[at:at + m], values), b
        at += m
    assert len({tuple(h) for h in history}) == n              # no two beams are alike
    s.close()
    s_all.close()
