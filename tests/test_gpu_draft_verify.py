"""Verification of drafted tokens (Serve.verify) against the sequential 64-bit
form: chains and trees, with and without draft rows, all types, odd
vocabularies, refused and repeated tokens, residuals of nothing, ties, bad
inputs; and that what it draws has the target's distribution."""
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


class Case:
    def __init__(self, nodes, vocab, tree, draft, dtype=torch.float32, seed=0, sharp=2.0):
        print(f"verify nodes={nodes[:8]} vocab={vocab} tree={tree} draft={draft} {dtype} seed={seed}", flush=True)
        r = np.random.default_rng(seed)
        T = sum(nodes)
        logits = sharp * r.standard_normal((T, vocab))
        soft = lambda x: np.exp(x - x.max(1, keepdims=True)) / np.exp(x - x.max(1, keepdims=True)).sum(1, keepdims=True)  # noqa: E731
        self.p = torch.from_numpy(soft(logits)).to(dtype)
        self.q = torch.from_numpy(soft(logits + r.standard_normal((T, vocab)))).to(dtype) if draft else None
        self.nodes, self.vocab, self.tree = nodes, vocab, tree
        self.parents, self.tokens = [], []
        at = 0
        for n in nodes:
            par = [-1] + [int(r.integers(max(0, j - 4), j)) if tree else j - 1 for j in range(1, n)]
            rows = (self.q if draft else self.p).double().numpy()
            for j in range(n):
                row = rows[at + max(par[j], 0)]
                self.tokens.append(int(r.choice(vocab, p=row / row.sum())))
            self.parents.append(par[:n])
            at += n
        self.u = torch.from_numpy(r.random(T)).float()
        self.race = torch.from_numpy(1 / r.exponential(size=(len(nodes), vocab))).float()
        self.q_start = torch.tensor(np.concatenate([[0], np.cumsum(nodes)]), dtype=torch.int32)

    def run(self, cap=None, serve=None):
        own = serve is None
        serve = serve or Serve(1, max(sum(self.nodes), 1), len(self.nodes))
        par = torch.tensor([p for ps in self.parents for p in ps], dtype=torch.int32, device=DEV) if self.tree else None
        got = serve.verify(self.p.to(DEV), torch.tensor(self.tokens, dtype=torch.int32, device=DEV), self.q_start.to(DEV), self.u.to(DEV), self.race.to(DEV),
                           draft_probs=None if self.q is None else self.q.to(DEV), parents=par, max_path=cap or max(max(self.nodes), 1))
        torch.cuda.synchronize()
        if own:
            assert serve.device_errors() == 0
            serve.close()
        return [t.cpu().numpy() for t in got]

    def check(self, path, count, tokens, cap=None):
        cap = cap or max(max(self.nodes), 1)
        at = 0
        for b, n in enumerate(self.nodes):
            if n == 0:
                assert count[b] == 0 and (path[b] == -1).all() and (tokens[b] == -1).all()
                continue
            s = slice(at, at + n)
            want, nxt, margin = R.verify(self.p[s].double().numpy(), None if self.q is None else self.q[s].double().numpy(), self.tokens[s], self.parents[b],
                                         self.u[s].double().numpy(), self.race[b].double().numpy(), min(cap, n))
            assert margin > 1e-5, "an input whose decision fp32 cannot be held to"
            fill = [-1] * (cap - len(want))
            assert count[b] == len(want) and path[b].tolist() == want + fill and tokens[b].tolist() == nxt + fill, b
            at += n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("nodes,vocab", [([1, 5, 3, 0, 9], 37), ([4, 2], 4099), ([16, 7, 1], 20011), ([6], 1)])
def test_against_the_sequential_form(nodes, vocab, tree, draft, dtype):
    c = Case(nodes, vocab, tree, draft, dtype, seed=vocab + 2 * tree + draft)
    c.check(*c.run())


@pytest.mark.parametrize("draft", [False, True])
def test_a_long_tree_and_a_short_path(draft):
    c = Case([150, 70], 500, True, draft, seed=21, sharp=0.5)
    c.check(*c.run())
    c.check(*c.run(cap=2), cap=2)
    c.check(*c.run(cap=1), cap=1)


def test_the_state_between_calls_is_clean():
    s = Serve(1, 40, 4)
    for seed in range(6):
        c = Case([3, 8, 1], 9001, bool(seed & 1), bool(seed & 2), seed=30 + seed)
        c.check(*c.run(serve=s))
    assert s.device_errors() == 0
    s.close()


def test_a_draft_equal_to_the_target_is_taken():
    c = Case([6, 6], 1000, False, True, seed=4)
    c.q = c.p.clone()
    path, count, tokens = c.run()
    assert (count == 6).all()


def test_refused_and_repeated_tokens_without_draft_rows():
    """The same token under two children: refused once, it has no probability left and is never drawn."""
    c = Case([4], 8, True, False, seed=5)
    c.parents = [[-1, 0, 0, 0]]
    c.p[0] = torch.tensor([0.5, 0.25, 0.125, 0.125, 0, 0, 0, 0])
    c.tokens = [0, 0, 0, 1]
    c.u = torch.tensor([0.0, 0.6, 0.0, 0.6])               # 0.6 >= 0.5; 0 < 0 fails; 0.6 * 0.5 >= 0.25
    c.race = torch.tensor([[9.0, 9.0, 1.0, 2.0, 50.0, 50.0, 50.0, 50.0]])
    path, count, tokens = c.run()
    assert count[0] == 1 and tokens[0, 0] == 3


def test_a_residual_of_nothing_falls_back_and_ties_go_to_the_lowest_index():
    c = Case([2, 1], 6000, False, True, seed=6)
    c.p[:] = 1 / 8192
    c.q[:] = 1 / 4096                                       # p < q everywhere: the residual is zero
    c.u[:] = 0.9
    c.race[:] = 1.0
    path, count, tokens = c.run()
    assert count.tolist() == [1, 1] and tokens[:, 0].tolist() == [0, 0]
    c.race[0, 4321] = 2.0
    c.race[0, 5999] = 2.0
    assert c.run()[2][0, 0] == 4321


def test_zero_negative_and_nan_probabilities():
    c = Case([1, 1], 3000, False, False, seed=7)
    c.p[0] = -1.0
    c.p[0, 17] = float("nan")
    c.p[0, 2999] = 1e-30
    s = Serve(1, 2, 2)
    assert c.run(serve=s)[2][0, 0] == 2999 and s.device_errors() == 0
    c.p[0] = 0.0
    out = c.run(serve=s)
    assert s.device_errors() == 8 and out[1].tolist() == [1, 1]
    s.close()


@pytest.mark.parametrize("draft", [False, True])
def test_bad_nodes_are_never_taken(draft):
    c = Case([4, 3], 50, True, draft, seed=8)
    s = Serve(1, 7, 2)
    good = [list(p) for p in c.parents], list(c.tokens)
    for what, at, value in (("tokens", 2, 50), ("tokens", 2, -3), ("parents", 2, 2), ("parents", 3, 9), ("parents", 1, -1)):
        c.parents, c.tokens = [list(p) for p in good[0]], list(good[1])
        c.u[:] = 0.0
        if what == "tokens":
            c.tokens[at] = value
        else:
            c.parents[0][at] = value
        path, count, tokens = c.run(serve=s)
        assert s.device_errors() == 4 and at not in path[0].tolist()[1:]
    s.close()


def test_bounds_outside_the_call_set_a_flag():
    c = Case([3, 3], 50, False, False, seed=9)
    s = Serve(1, 6, 2)
    for starts in ([0, 3, 7], [0, -1, 6], [0, 5, 3]):
        c.q_start = torch.tensor(starts, dtype=torch.int32)
        c.run(serve=s)
        assert s.device_errors() & 1
    s.close()


def test_strided_rows():
    c = Case([3, 5], 1001, True, True, seed=10)
    want = c.run()
    p = torch.full((8, 2100), float("nan"), device=DEV)
    p[:, 3:1004] = c.p.to(DEV)
    q = torch.full((8, 1500), float("nan"), device=DEV)
    q[:, :1001] = c.q.to(DEV)
    race = torch.full((2, 1003), float("nan"), device=DEV)
    race[:, 1:1002] = c.race.to(DEV)
    s = Serve(1, 8, 2)
    par = torch.tensor([x for y in c.parents for x in y], dtype=torch.int32, device=DEV)
    got = s.verify(p[:, 3:1004], torch.tensor(c.tokens, dtype=torch.int32, device=DEV), c.q_start.to(DEV), c.u.to(DEV), race[:, 1:1002], draft_probs=q[:, :1001], parents=par, max_path=5)
    for a, b in zip(got, want):
        assert np.array_equal(a.cpu().numpy(), b)
    s.close()


@pytest.mark.parametrize("draft", [False, True])
def test_what_is_drawn_follows_the_target(draft):
    """20000 one-step drafts from one draft row: the first token's frequencies
    are the target's within five standard deviations of each."""
    n, vocab = 20000, 7
    r = np.random.default_rng(11)
    p = np.array([0.3, 0.05, 0.2, 0.1, 0.15, 0.12, 0.08])
    q = np.array([0.1, 0.3, 0.1, 0.2, 0.1, 0.1, 0.1])
    x = r.choice(vocab, size=n, p=q) if draft else np.full(n, 2)
    tokens = np.stack([np.zeros(n, int), x], 1).reshape(-1)
    P = torch.from_numpy(np.tile(p, (2 * n, 1))).float().to(DEV)
    Q = torch.from_numpy(np.tile(q, (2 * n, 1))).float().to(DEV) if draft else None
    s = Serve(1, 2 * n, n)
    _, _, nxt = s.verify(P, torch.from_numpy(tokens).int().to(DEV), (2 * torch.arange(n + 1)).int().to(DEV), torch.from_numpy(r.random(2 * n)).float().to(DEV),
                         torch.from_numpy(1 / r.exponential(size=(n, vocab))).float().to(DEV), draft_probs=Q, max_path=2)
    got = np.bincount(nxt[:, 0].cpu().numpy(), minlength=vocab) / n
    assert np.all(np.abs(got - p) <= 5 * np.sqrt(p * (1 - p) / n)), got
    s.close()


def test_refusals():
    s = Serve(1, 4, 2)
    p = torch.full((2, 8), 0.125, device=DEV)
    t, u = torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros(2, device=DEV)
    st, race = torch.tensor([0, 2], dtype=torch.int32, device=DEV), torch.ones(1, 8, device=DEV)
    s.verify(p, t, st, u, race)
    for args, kw in (((p.double(), t, st, u, race), {}), ((p, t.long(), st, u, race), {}), ((p, t, st, u.double(), race), {}), ((p, t, st, u, race[:, :4]), {}),
                     ((p, t, st, u, race), dict(draft_probs=p.half())), ((p, t, st, u, race), dict(parents=t[:1])), ((p, t, st, u, race), dict(max_path=0)),
                     ((p.t().contiguous().t(), t, st, u, race), {})):
        with pytest.raises((TypeError, ValueError)):
            s.verify(*args, **kw)
    many = torch.zeros(5, 8, device=DEV)
    with pytest.raises(B.ColiError) as e:
        s.verify(many, torch.zeros(5, dtype=torch.int32, device=DEV), st, torch.zeros(5, device=DEV), race)
    assert e.value.status == B.E_INVALID
    s.close()
