"""tfl_beam_select in calls of many rows, whose CTAs have 256 threads where those of small calls have 512: a search's ranking is
that of the search alone, down to scores that differ in their 64-bit sums' last bits alone."""
import pytest
import torch

from gqa_decoder_forward_gb300 import build, tfl
from tests.test_gpu_beam_select import BIG, normal, outputs, plain_model

pytestmark = pytest.mark.gpu
CHUNKS = (BIG.vocab + 8191) // 8192


@pytest.fixture(scope="module")
def big():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    build.build()
    return plain_model(BIG, 64)


@pytest.mark.parametrize("seed", range(8))
def test_near_ties_do_not_depend_on_the_rest_of_the_call(big, seed):
    """Beams whose rows hold the same numbers in different orders: equal scores but for what sums round."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    beams = min(16, sms // CHUNKS)                # alone: a CTA per SM at most
    groups = 64 // beams
    assert beams >= 2 and groups * beams * CHUNKS > sms
    gen = torch.Generator(device="cuda").manual_seed(630 + seed)
    rows = normal(640 + seed, groups, BIG)
    z = torch.stack([row[torch.randperm(BIG.vocab, generator=gen, device="cuda")] for row in rows for _ in range(beams)])
    scores = torch.zeros(groups, beams, device="cuda")
    whole = outputs(groups, 32, True)
    tfl.tfl_beam_select(big, z, scores, **whole)
    for g in range(groups):
        alone = outputs(1, 32, True)
        tfl.tfl_beam_select(big, z[g * beams: (g + 1) * beams], scores[g: g + 1], **alone)
        assert torch.equal(alone["ids"][0], whole["ids"][g])
        assert torch.equal(alone["parents"][0] + g * beams, whole["parents"][g])
        assert torch.equal(alone["out_scores"][0], whole["out_scores"][g])
    assert big.status() == tfl.TFL_OK
