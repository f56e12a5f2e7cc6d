"""Beam selection where logits and scores are far from ordinary ones: tokens masked with large negative values of
their type, single large logits, rows far from zero, and every kind of NaN, in vocabularies of either chunk size."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from int4_routed_expert_layer_amd.serve import Serve  # noqa: E402
from test_gpu_beam import DEV, TYPE  # noqa: E402

SIZES = [(1, 3, 5000), (8, 8, 9001)]                          # chunks of 2048 and of 8192 logits


def select(logits, scores, keep):
    """logits [g, b, v], scores [g, b] -> scores, parents, tokens [g, keep] in 64 bits.  A token's distance from its row's
    greatest logit comes first: of large logits it would swallow what is added to it."""
    g, b, v = logits.shape
    out = np.full((g, keep), -np.inf), np.full((g, keep), -1), np.full((g, keep), -1)
    for i in range(g):
        found = []
        for j in range(b):
            z = np.where(np.isnan(logits[i, j]), -np.inf, logits[i, j])
            top = z.max()
            if not np.isfinite(scores[i, j]) or not np.isfinite(top):
                continue
            total = (scores[i, j] - np.log(np.exp(z - top).sum())) + (z - top)
            best = np.lexsort((np.arange(v), -z))[:keep]
            found += [(-total[t], j, -z[t], t) for t in best if np.isfinite(z[t])]
        for r, (s, j, _, t) in enumerate(sorted(found)[:keep]):
            out[0][i, r], out[1][i, r], out[2][i, r] = -s, j, t
    return out


def check(logits, scores, keep):
    """Scores are off by their rounding to fp32 and by the logarithm of a sum of fp32 exponentials: of each the exponent is off
    by 2^-24 of itself (24 at most where it counts), the exponential by two units more, and a thread's sum of 32 terms by 32:
    2^-24 (24 + 2 + 32 + 8)."""
    g, b, v = logits.shape
    s = Serve(1, 1, g * b)
    want = select(logits.double().numpy(), scores.double().numpy(), keep)
    best, parents, tokens = (x.cpu().numpy() for x in s.beam_select(logits.view(g * b, v).to(DEV), scores.to(DEV), keep))
    assert s.device_errors() == 0
    s.close()
    assert np.array_equal(parents, want[1]) and np.array_equal(tokens, want[2])
    live = parents >= 0
    assert np.all(np.isneginf(best[~live]))
    assert np.all(np.abs(best[live] - want[0][live]) <= 2.0 ** -24 * (66 + np.abs(want[0][live])))


def normal(g, b, v, kind, seed):
    r = torch.Generator().manual_seed(seed)
    return (3 * torch.randn(g, b, v, generator=r)).to(TYPE[kind]), -4 * torch.rand(g, b, generator=r)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("value", [-1e9, -6e9, -1e10, -1e12, -1e20, -1e30, -3e38])
@pytest.mark.parametrize("g,b,v", SIZES)
def test_tokens_masked_with_a_large_value(g, b, v, value, kind):
    """A constraint that leaves few tokens: waves and whole chunks hold nothing but masked ones."""
    logits, scores = normal(g, b, v, kind, 11)
    logits[:, :, 7:] = value
    check(logits, scores, 8)
    check(logits, scores, 20)                                 # masked tokens follow where there are no others
    logits, scores = normal(g, b, v, kind, 12)
    logits[:, :, :v - 300] = value
    check(logits, scores, 16)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("value", [1e9, 6e9, 1e10, 1e20, 1e30, 3e38])
@pytest.mark.parametrize("g,b,v", SIZES)
def test_single_large_logits(g, b, v, value, kind):
    """The token that holds it has all the probability; what follows is as far behind as the logits are apart."""
    logits, scores = normal(g, b, v, kind, 13)
    logits[:, 0, 3], logits[:, b - 1, v - 1] = value, value
    check(logits, scores, 2)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("value", [-1e10, -1e12, -1e20, -3e38, 1e9, 1e20, 3e38])
@pytest.mark.parametrize("g,b,v", SIZES)
def test_rows_that_lie_far_from_zero(g, b, v, value, kind):
    """Rows of one large value each: every token of a row has the same share of its beam's score, whatever the value."""
    logits, scores = normal(g, b, v, kind, 16)
    logits[:, 0], logits[:, b - 1] = value, -value / 4
    check(logits, scores, 12)
    scores[:, 0] += 8
    check(logits, scores, 12)


@pytest.mark.parametrize("g,b,v", SIZES)
def test_the_largest_logits_of_f16(g, b, v):
    logits, scores = normal(g, b, v, "f16", 14)
    logits[:, :, 5:] = -65504
    check(logits, scores, 5)
    logits[:, :, 4] = 65504
    check(logits, scores, 2)


@pytest.mark.parametrize("kind,bits", [("f32", (0x7F800001, 0x7FC00000, 0x7FFFFFFF)), ("bf16", (0x7F81, 0x7FC0, 0x7FFF)), ("f16", (0x7C01, 0x7E00, 0x7FFF))])
@pytest.mark.parametrize("g,b,v", SIZES)
def test_every_nan_counts_as_minus_infinity(g, b, v, kind, bits):
    logits, scores = normal(g, b, v, kind, 15)
    raw = logits.view(torch.int32 if kind == "f32" else torch.int16)
    sign = -(1 << (31 if kind == "f32" else 15))
    for i, x in enumerate(bits):
        raw[:, :, 2 * i::11] = x
        raw[:, :, 2 * i + 1::11] = x + sign
    check(logits, scores, 9)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("low", [-1e9, -1e20, -1e30])
@pytest.mark.parametrize("g,b,v", SIZES)
def test_scores_that_swallow_the_logits(g, b, v, low, kind):
    """Beams that begin with a very low score in place of -inf: the 64-bit scores of their tokens coincide, but within a beam
    the greater logit still comes first; equal scores of different beams go by the beam."""
    logits, scores = normal(g, b, v, kind, 17)
    scores[:] = low
    check(logits, scores, 9)
    scores[:, 0] = -1
    logits[:, 0, 4:] = -float("inf")                          # four tokens of the first beam, then those of others
    check(logits, scores, 12)
    logits = (1 + torch.arange(v).remainder(89) * 2.0 ** -23).expand(g, b, v).contiguous().to(TYPE[kind])
    check(logits, scores, 12)                                 # neighbours in fp32
