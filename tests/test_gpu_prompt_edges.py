"""Expanded latent attention (Serve.prompt): bounds of sequences past the first 64,
and prompts whose keys are divided into two rounds of parts."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_latent_prompt import DEV, HEADS, Case  # noqa: E402
from int4_routed_expert_layer_amd.serve import Serve  # noqa: E402


@pytest.mark.parametrize("width", ["wide", "narrow"])
@pytest.mark.parametrize("n_seq,at", [(65, 64), (200, 63), (200, 130), (200, 199)])
@pytest.mark.parametrize("which", ["q", "k", "both"])
def test_bounds_of_any_sequence_set_the_flag(width, n_seq, at, which):
    """One token a sequence; the bounds of sequence `at` leave the call (the sequences after it begin where they end)."""
    nope, v = HEADS[width]
    g = torch.Generator().manual_seed(n_seq + at)
    starts = torch.arange(n_seq + 1, dtype=torch.int32)
    starts[at + 1:] -= 1                                    # sequence `at` is empty
    n = int(starts[-1])
    q = torch.randn(n, 2, nope + 64, generator=g).bfloat16().to(DEV)
    kv = torch.randn(n, 2, nope + v, generator=g).bfloat16().to(DEV)
    pe = torch.randn(n, 64, generator=g).bfloat16().to(DEV)
    s = Serve(2, n, n_seq, nope=nope, v_dim=v)
    good = s.prompt(q, kv, pe, starts.to(DEV), starts.to(DEV), 0.1)
    assert s.device_errors() == 0
    bad = starts.clone()
    bad[at + 1:] += 100000
    out = torch.zeros_like(good)
    s.prompt(q, kv, pe, (bad if which != "k" else starts).to(DEV), (bad if which != "q" else starts).to(DEV), 0.1, out=out)
    assert s.device_errors() == 1
    assert torch.equal(out[:at], good[:at])
    s.close()


@pytest.mark.parametrize("nq,nk,heads", [([1600], [1600], dict(wide=10, narrow=20)), ([1700], [2500], dict(wide=10, narrow=20)), ([1600, 1690], [1600, 1700], dict(wide=5, narrow=10))])
@pytest.mark.parametrize("width", ["wide", "narrow"])
def test_prompts_of_two_rounds_of_parts(width, nq, nk, heads):
    """At least 768 keys a sequence, fewer than twice the queries, and more than
    half a round of tiles: the keys are divided though one round would not divide them."""
    c = Case(nq, nk, heads[width], width, seed=21)
    out, lse = c.run()
    c.check(out, lse, heads=[0, heads[width] // 2, heads[width] - 1])
    again, again_lse = c.run()
    assert torch.equal(out, again) and torch.equal(lse, again_lse)
