"""Calls of the 8-bit cache's, prefix and beam operators at the edges of what they allow: bounds that do not ascend
where no row falls, other numbers of sequences than a workgroup looks at, a step planned beside calls that use the
same scratch, and long prefixes beside short sequences."""
import numpy as np
import pytest

import serve_case as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from int4_routed_expert_layer_amd.serve import Serve  # noqa: E402
from test_gpu_latent_cache import DEV  # noqa: E402
from test_gpu_latent8_cache import Paged, ints  # noqa: E402
from test_gpu_prefix_decode import Shared  # noqa: E402


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("n,at", [(3, 1), (300, 7), (300, 299), (5000, 4100)])
def test_read_flags_bounds_that_do_not_ascend_wherever_they_are(n, at, bits):
    """The first sequence holds all rows; a bound of a later one, that no row's search meets, lies before them."""
    p = Paged([20] + [0] * (n - 1), 16, "bf16", bits, seed=n)
    s = Serve(1, 1, n, 16)
    assert torch.equal(p.run(s, n=20).cpu(), p.want())
    assert s.device_errors() == 0
    p.k_start[at] = 25 if at < n - 1 else -3
    p.run(s, n=20)
    assert s.device_errors() & 1                             # and 2 where rows now fall to a sequence without pages
    s.close()


def test_selection_between_a_plan_and_its_decode():
    """beam_select uses the scratch of the partial results, which a decode fills and reads in one call: neither harms the other."""
    g = torch.Generator().manual_seed(1)
    s = Serve(16, 4, 4, 16)
    lens = [3000, 17, 900, 64]
    pages = [-(-n // 16) for n in lens]
    table = torch.full((4, max(pages)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    cache = torch.randn(at, 16, R.ROW, generator=g).bfloat16().to(DEV)
    ql, qp = torch.randn(4, 16, R.LATENT, generator=g).bfloat16().to(DEV), torch.randn(4, 16, R.ROPE, generator=g).bfloat16().to(DEV)
    logits, scores = torch.randn(4, 40000, generator=g).to(DEV), torch.zeros(1, 4, device=DEV)
    s.plan(ints(np.arange(5)), ints(lens), n_tok=4)
    want = s.decode(ql, qp, cache, table.to(DEV), 0.05)
    best = s.beam_select(logits, scores, 4)
    for _ in range(3):
        assert torch.equal(s.decode(ql, qp, cache, table.to(DEV), 0.05), want)
        assert all(torch.equal(a, b) for a, b in zip(s.beam_select(logits, scores, 4), best))
    assert s.device_errors() == 0
    s.close()


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("prefix,n,heads,own", [(9000, 40, 16, 700), (700, 260, 16, 130), (16500, 20, 64, 200)])
def test_long_prefixes_beside_short_sequences_of_few_rows(prefix, n, heads, own, bits):
    """Plans of more items than CUs whose long runs have a CU to themselves, and pieces of 32 rows or fewer."""
    r = np.random.default_rng(n)
    c = Shared([(prefix, [int(x) for x in r.integers(1, own, n)], [1] * n)], heads, 64, "f16", bits, seed=n)
    c.check(*c.run(), heads=[0, heads - 1])
