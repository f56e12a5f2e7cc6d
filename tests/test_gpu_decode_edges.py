"""Absorbed latent attention (Serve.decode): keys of infinite latents wherever
they lie, and captured calls whose plan has become another's."""
import numpy as np
import pytest

import serve_case as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_latent_decode import DEV, Case  # noqa: E402
from int4_routed_expert_layer_amd.serve import Serve  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("length,page", [(92, 16), (733, 1)])
@pytest.mark.parametrize("back", [82, 22, 5, 2, 1])
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_an_infinite_latent_that_a_row_sees(back, length, page, value, tree, dtype):
    """Column 9 of one cached row is infinite, in the context or in one of the
    five last positions, of one piece or of many.  A row that sees it with a query of the same sign has a
    score of +inf and is NaN; with the other sign the score is -inf, so the
    weight is zero and the column 0 * inf, NaN, while the rest is as if the key
    were not there.  A row that does not see it is as if it were not there."""
    heads, n, pos = 20, 5, length - back
    sets = [R.ancestors([-1, 0, 0, 1, 2])] if tree else None
    c = Case([length], [n], heads, page, dtype, sets=sets, seed=31)
    side = torch.where(torch.arange(heads) % 2 == 0, 1.0, -1.0)
    c.q[:, :, 9] = (side[None] * (0.5 + c.q[:, :, 9].float().abs())).to(c.q.dtype)
    c.cache[c.table[0, pos // page], pos % page, 9] = value
    out, lse = (x.double().cpu().numpy() for x in c.run())
    see, kv = c.seen(0), c.kv[0].double().numpy()
    others = np.arange(R.LATENT) != 9
    for h in range(heads):
        sees = see.copy()
        sees[:, pos] = False
        o, e, bo, be = R.attend(c.q[:, h].double().numpy(), kv, kv[:, :R.LATENT], sees, c.scale, dtype)
        for i in range(n):
            if not see[i, pos]:
                assert np.all(np.abs(out[i, h] - o[i]) <= bo[i]) and abs(lse[i, h] - e[i]) <= be[i], (i, h)
            elif side[h] * value > 0:
                assert np.isnan(out[i, h]).all() and np.isnan(lse[i, h]), (i, h)
            else:
                assert np.isnan(out[i, h, 9]), (i, h)
                assert np.all(np.abs(out[i, h] - o[i])[others] <= bo[i][others]) and abs(lse[i, h] - e[i]) <= be[i], (i, h)


@pytest.mark.parametrize("lens,nodes", [([600, 90], [2, 1]), ([40, 40], [1, 1])])
@pytest.mark.parametrize("more", [([5000, 300], [3, 6]), ([50, 3000, 700], [1, 1, 1])])
def test_a_captured_call_after_a_larger_plan(lens, nodes, more):
    """A call captured for few tokens and replayed when the handle holds the plan
    of a larger step: a flag, and nothing is read or written; with its own plan again, its own result."""
    c = Case(lens, nodes, 16, 16, seed=41)
    want, want_lse = c.run()
    n, T = sum(nodes), sum(more[1])
    s = Serve(16, T, len(more[0]), 16)
    q, cache, table = c.q.to(DEV), c.cache.to(DEV), c.table.to(DEV)
    ql, qp = q[..., :R.LATENT].contiguous(), q[..., R.LATENT:].contiguous()
    own = c.q_start.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    other = torch.tensor(np.concatenate([[0], np.cumsum(more[1])]), dtype=torch.int32, device=DEV), torch.tensor(more[0], dtype=torch.int32, device=DEV)
    room, room_lse = torch.empty(T, 16, R.LATENT, dtype=torch.bfloat16, device=DEV), torch.empty(T, 16, device=DEV)
    out, lse = room[:n], room_lse[:n]
    s.plan(*own, n_tok=n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.decode(ql, qp, cache, table, c.scale, out=out, lse=lse)
    for _ in range(2):
        room.fill_(7.0)
        room_lse.fill_(7.0)
        s.plan(*other, n_tok=T)
        graph.replay()
        assert s.device_errors() == 1
        assert torch.all(room == 7.0) and torch.all(room_lse == 7.0)
        s.plan(*own, n_tok=n)
        graph.replay()
        assert s.device_errors() == 0
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    s.close()


@pytest.mark.parametrize("lens,nodes,heads", [([5000], [1], 64), ([2000, 17, 900, 1], [2, 1, 3, 1], 33), ([150] * 300, [1] * 300, 16), ([700] * 5, [20] * 5, 64), ([1500], [40], 64)])
def test_every_row_of_divided_and_many_units(lens, nodes, heads):
    """All heads of all tokens: each 64-row unit has pieces and a join of its own."""
    c = Case(lens, nodes, heads, 32, seed=51)
    c.check(*c.run())
