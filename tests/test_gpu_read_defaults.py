"""Serve.read as it is called without its optional arguments: positions from 0, and as many rows as the bounds say, or as
an output tensor has; with and without first positions no flag is set."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import serve_case as R  # noqa: E402
from int4_routed_expert_layer_amd.serve import Serve  # noqa: E402
from test_gpu_latent8_cache import DEV, Paged, ints  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("lens,page,first", [([1], 1, [0]), ([17, 0, 0, 33, 1, 100], 16, [0] * 6), ([15, 16, 17, 48], 4, [3, 0, 7, 61]), ([0, 0, 5], 64, [200, 1, 0]),
                                             ([3] * 70 + [0] * 130 + [2] * 9, 2, [5] * 209), ([1000], 64, [23])])
def test_read_from_first_positions_and_from_the_beginning(lens, page, first, bits, dtype):
    p = Paged(lens, page, dtype, bits, seed=len(lens) + 1, first=first)
    s = Serve(1, 1, len(lens), page, dtype=dtype)
    cache, table, k_start = p.cache.to(DEV), p.table.to(DEV), p.k_start.to(DEV)
    assert torch.equal(s.read(cache, table, k_start, first=ints(first)).cpu(), p.want())
    assert s.device_errors() == 0
    p.first = [0] * len(lens)
    want = p.want()
    assert len(want) == sum(lens) > 0
    assert torch.equal(s.read(cache, table, k_start).cpu(), want)
    out = torch.full((sum(lens) + 3, R.ROW), 7.0, dtype=want.dtype, device=DEV)
    assert s.read(cache, table, k_start, out=out) is out
    assert torch.equal(out[:-3].cpu(), want) and torch.all(out[-3:] == 7)
    assert s.device_errors() == 0
    s.close()
