"""Verification of drafted tokens (Serve.verify) where a call has no nodes, and
where probabilities are negative or NaN (they count as zero)."""
import numpy as np
import pytest

import serve_case as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_draft_verify import DEV, Case  # noqa: E402
from int4_routed_expert_layer_amd import binding as B  # noqa: E402
from int4_routed_expert_layer_amd.serve import Serve  # noqa: E402


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("starts,flags", [([0, 0, 0, 0], 0), ([0, 0, 2, 2], 1)])
def test_a_call_without_nodes(kind, starts, flags):
    """n_tok = 0: no probabilities, tokens or random numbers are needed (NULL), and every path is empty."""
    s = Serve(1, 4, 3)
    q_start = torch.tensor(starts, dtype=torch.int32, device=DEV)
    for cols, draft in ((1, False), (5, True)):
        path, nxt = (torch.full((3, cols), 7, dtype=torch.int32, device=DEV) for _ in range(2))
        count = torch.full((3,), 7, dtype=torch.int32, device=DEV)
        parents = q_start.data_ptr() if draft else None     # never read
        st = B.lib.coli_draft_verify(s.handle, None, 0, None, 0, kind, 50000, None, parents, q_start.data_ptr(), 3, 0, None, None, 0,
                                     path.data_ptr(), cols, count.data_ptr(), nxt.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert st == B.OK and s.device_errors() == flags
        assert (path == -1).all() and (nxt == -1).all() and (count == 0).all()
    c = Case([3, 1, 0], 500, True, True, seed=3)             # the handle serves ordinary calls as before
    c.check(*c.run(serve=s))
    s.close()


BAD = [float("nan"), -0.5, -float("inf")]


def clip(x):
    x = x.double().numpy()
    return np.where(x > 0, x, 0.0)


def expect(c, path, count, tokens):
    """The sequential form on the clipped rows."""
    cap, at = max(c.nodes), 0
    for b, n in enumerate(c.nodes):
        s = slice(at, at + n)
        want, nxt, margin = R.verify(clip(c.p[s]), None if c.q is None else clip(c.q[s]), c.tokens[s], c.parents[b], c.u[s].double().numpy(), c.race[b].double().numpy(), n)
        assert margin > 1e-5, "an input whose decision fp32 cannot be held to"
        fill = [-1] * (cap - len(want))
        assert count[b] == len(want) and path[b].tolist() == want + fill and tokens[b].tolist() == nxt + fill, b
        at += n


@pytest.mark.parametrize("bad", BAD)
def test_a_sibling_of_no_probability_without_draft_rows(bad):
    """Two children of the root: the first one's probability is no number above zero, so the second is tried against 0.5."""
    c = Case([3], 4, True, False, seed=1)
    c.parents, c.tokens = [[-1, 0, 0]], [0, 0, 1]
    c.p[0] = torch.tensor([bad, 0.5, 0.3, 0.2])
    c.u = torch.tensor([0.0, 0.5, 0.4])
    path, count, tokens = c.run()
    assert path[0].tolist() == [0, 2, -1] and count[0] == 2 and tokens[0, 0] == 1


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("tree", [False, True])
def test_draft_probabilities_of_no_value(bad, tree):
    """q of the drafted token counts as zero: taken where the target has it, refused where it has not."""
    c = Case([2], 4, tree, True, seed=2)
    c.parents, c.tokens = [[-1, 0]], [0, 1]
    c.q[0] = torch.tensor([0.5, bad, 0.25, 0.25])
    c.u = torch.tensor([0.0, 0.9])
    c.p[0] = torch.tensor([0.5, 0.25, 0.25, 0.0])
    assert c.run()[1][0] == 2
    c.p[0] = torch.tensor([0.25, 0.0, 0.25, 0.5])
    c.race[:] = 1.0
    path, count, tokens = c.run()
    assert count[0] == 1 and tokens[0, 0] == 3                # of (p - q)+ = 0, 0, 0, 0.25


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("vocab", [41, 4099])
def test_negative_and_nan_probabilities_count_as_zero(vocab, draft, tree, dtype):
    """A part of every row, drafted tokens among them, has no value above zero."""
    c = Case([9, 12, 3, 7], vocab, tree, draft, dtype, seed=50 + 2 * tree + draft)
    r = np.random.default_rng(vocab)
    bad = torch.tensor(BAD, dtype=dtype)
    for rows in [c.p] + ([c.q] if draft else []):
        for t in range(len(rows)):
            at = r.choice(vocab, vocab // 8, replace=False)
            rows[t, torch.from_numpy(at)] = bad[torch.from_numpy(r.integers(0, 3, len(at)))]
        at = 0
        for ps, n in zip(c.parents, c.nodes):
            for j in range(1, n):
                if r.random() < 0.4:
                    rows[at + ps[j], c.tokens[at + j]] = bad[int(r.integers(0, 3))]
            at += n
    expect(c, *c.run())
