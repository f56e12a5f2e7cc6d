"""Verification of drafted tokens (Serve.verify) where a call has no nodes."""
import pytest

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
