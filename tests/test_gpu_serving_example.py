"""The serving operators, the expert layer and a paged cache put together as in
examples/serving_step.py: both forms of attention agree on one prompt, and the
cache after speculative steps holds the generated sequence's rows."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import serving_step as E  # noqa: E402

U = 2.0 ** -8      # unit roundoff of bf16


@pytest.fixture(scope="module")
def model():
    m = E.Model(seed=3)
    yield m
    m.close()


def test_the_two_forms_of_attention_agree(model):
    """A prompt of 45 tokens expanded, and as a chain over its own cache rows.
    Between them lie one rounding of keys, values, absorbed queries and latent
    outputs each: scores differ by up to 2 u sum|q k| scale (about 3 here), so
    weights by 2.4%, and outputs by that share of the largest value, twice."""
    n, dev = 45, model.device
    tokens = E.ints([(7 * i) % E.VOCAB for i in range(n)], dev)
    cache = torch.zeros(3, E.PAGE, E.ROW, dtype=torch.bfloat16, device=dev)
    slots, starts = torch.arange(n, device=dev), E.ints([0, n], dev)
    seen = {}

    def keep(name, attend):
        def run(q_nope, q_pe):
            seen[name] = attend(q_nope, q_pe)
            return seen[name]
        return run

    pos = torch.arange(n, device=dev, dtype=torch.int32)
    model.layer(tokens, pos, slots, cache, keep("expanded", model.expanded(slots, cache, starts)))
    model.serve.plan(starts, E.ints([n], dev), n_tok=n)
    model.layer(tokens, pos, slots, cache, keep("absorbed", model.absorbed(cache, E.ints([[0, 1, 2]], dev))))
    a, b = seen["expanded"].float(), seen["absorbed"].float()
    assert torch.isfinite(a).all() and (a - b).abs().max() <= 0.05 * a.abs().max()


def test_the_cache_holds_the_generated_sequence(model):
    tokens, accepted, rows = E.generate(model, list(range(3, 40)), 10, seed=5)
    assert len(rows) == len(tokens) - 1 == 36 + sum(accepted) + 10
    assert sum(accepted) > 0, "the drafter should have some of its tokens accepted"
    n, dev = len(rows), model.device
    fresh = torch.zeros(-(-n // E.PAGE), E.PAGE, E.ROW, dtype=torch.bfloat16, device=dev)
    h = E.rms(model.embed[torch.tensor(tokens[:n], device=dev)])
    model.serve.append(h @ model.w_kv, model.kv_norm, E.EPS, model.cos, model.sin, torch.arange(n, device=dev, dtype=torch.int32), torch.arange(n, device=dev), fresh)
    want = fresh.view(-1, E.ROW)[:n].float()
    # The projection rounds once and the row once more, in either batch.
    assert ((rows.float() - want).abs() <= 4 * U * want.abs().amax(1, keepdim=True)).all()


def test_generation_repeats(model):
    first = E.generate(model, [5, 9, 2], 6, seed=8)
    again = E.generate(model, [5, 9, 2], 6, seed=8)
    assert first[0] == again[0] and first[1] == again[1] and torch.equal(first[2], again[2])
