"""Old and new block tables of Serve.beam_reorder in one tensor: row beside row they share nothing and are both whole;
tables that have an element in common are refused."""
import numpy as np
import pytest

import serve8_case as R8

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from int4_routed_expert_layer_amd import binding as B  # noqa: E402
from int4_routed_expert_layer_amd.serve import Serve  # noqa: E402
from test_gpu_beam import DEV, Beams, ints  # noqa: E402

PARENTS = [[1, 1, 3, 1], [0, 2, 2, 0]]


def both(b, at, out_at, width):
    """A tensor with the table from column `at` on, and its parts for the old and the new one."""
    cols = b.table.shape[1]
    wide = torch.full((8, width), -7, dtype=torch.int32, device=DEV)
    wide[:, at:at + cols] = b.table.to(DEV)
    return wide, wide[:, at:at + cols], wide[:, out_at:out_at + cols]


@pytest.mark.parametrize("gap", [0, 3])
@pytest.mark.parametrize("first", ["old", "new"])
def test_tables_that_lie_row_beside_row(first, gap):
    b = Beams([37, 20], 4, 16, 1, 16, seed=21)
    cols = b.table.shape[1]
    at, out_at = (0, cols + gap) if first == "old" else (cols + gap, 0)
    s = Serve(1, 1, 8, 16)
    wide, table, out = both(b, at, out_at, 2 * cols + gap)
    cache = b.cache.to(DEV)
    s.beam_reorder(cache, table, ints(np.repeat(b.lens, 4)), ints(PARENTS), out=out)
    assert s.device_errors() == 0
    want_cache, want_table = R8.reorder(b.cache, b.table, b.lens, np.asarray(PARENTS), 16)
    assert torch.equal(out.cpu(), want_table) and torch.equal(table.cpu(), b.table)
    assert torch.equal(cache.cpu(), want_cache)
    if gap:
        assert torch.all(wide[:, cols:cols + gap] == -7)
    s.close()


def test_tables_with_an_element_in_common_are_refused():
    b = Beams([37, 20], 4, 16, 1, 16, seed=22)
    cols = b.table.shape[1]
    s = Serve(1, 1, 8, 16)
    cache, lens, parents = b.cache.to(DEV), ints(np.repeat(b.lens, 4)), ints(PARENTS)
    # one column in common, on either side; a row further; all; of rows that lie apart by different strides
    flat = torch.zeros(64 * cols, dtype=torch.int32, device=DEV)
    size = (8, cols)
    cases = [(0, cols - 1, 2 * cols), (cols - 1, 0, 2 * cols), (0, cols + 1, 2 * cols), (0, 2 * cols + cols - 1, 2 * cols), (5, 5, 2 * cols)]
    pairs = [(flat.as_strided(size, (w, 1), x), flat.as_strided(size, (w, 1), y)) for x, y, w in cases]
    pairs.append((flat.as_strided(size, (2 * cols, 1), 0), flat.as_strided(size, (3 * cols, 1), cols)))
    for table, out in pairs:
        with pytest.raises(B.ColiError) as e:
            s.beam_reorder(cache, table, lens, parents, out=out)
        assert e.value.status == B.E_INVALID and "overlap" in str(e.value)
    s.close()
