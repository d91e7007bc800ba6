"""tfl_beam_select in calls of many rows, whose CTAs have 256 threads where those of small calls have 512: a search's ranking is
that of the search alone, down to scores that differ in their 64-bit sums' last bits alone.  And the numbers, masks and flags of
test_gpu_beam_select in such calls, with its tolerance (its bound is that of 32 logits added up by a thread)."""
import numpy as np
import pytest
import torch

from gqa_decoder_forward_gb300 import build, tfl
from tests.test_gpu_beam_select import BIG, KINDS, check, normal, outputs, plain_model, rows_like, scores_of

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


def large_call(rows):
    """How often `rows` rows are repeated so that there are more chunks than SMs."""
    groups = torch.cuda.get_device_properties(0).multi_processor_count // (rows * CHUNKS) + 1
    assert groups * rows <= 64
    return groups


@pytest.mark.parametrize("kind", KINDS)
def test_distributions(big, kind):
    z = rows_like(kind, BIG.vocab).to(torch.bfloat16).cuda()
    groups = large_call(4)
    scores = torch.tensor([[-3.0, -3.0, -5.0, -3.0]], device="cuda").repeat(groups, 1)
    for n_out in (32, 1):
        out = check(big, z.repeat(groups, 1), scores, n_out)
        assert all(torch.equal(out["out_scores"][0], o) for o in out["out_scores"])


@pytest.mark.parametrize("allowed", [0, 1, 2, 31, 33, 700, 3000])
def test_masked_vocabulary(big, allowed):
    z = normal(650, 3, BIG)
    keep = torch.zeros(BIG.vocab, dtype=torch.bool, device="cuda")
    keep[8190: 8190 + allowed] = True
    z[0, ~keep] = float("-inf")
    z[1, ~keep.roll(3)] = float("-inf")
    groups = large_call(3)
    check(big, z.repeat(groups, 1), scores_of(651, groups, 3), 32)
    groups = large_call(2)
    check(big, z[:2].repeat(groups, 1), scores_of(652, groups, 2), 32)
    check(big, z[:2].repeat(groups, 1), scores_of(653, 2 * groups, 1), 5)


@pytest.mark.parametrize("allowed", [1, 7, 40])
def test_a_few_ids_anywhere(big, allowed):
    """A grammar's mask: some ids of the whole vocabulary, most chunks without one."""
    gen = torch.Generator(device="cuda").manual_seed(654)
    groups = large_call(4)
    z = torch.full((4 * groups, BIG.vocab), float("-inf"), dtype=torch.bfloat16, device="cuda")
    for row, values in zip(z, normal(655, 4 * groups, BIG)):
        at = torch.randperm(BIG.vocab, generator=gen, device="cuda")[:allowed]
        row[at] = values[at]
    check(big, z, scores_of(656, groups, 4), 32)
    check(big, z[:4].contiguous(), scores_of(656, 1, 4), 32)


def test_lowest_values_are_not_masks(big):
    groups = large_call(2)
    z = torch.full((2, BIG.vocab), torch.finfo(torch.bfloat16).min, dtype=torch.bfloat16, device="cuda")
    z[0, 17] = z[0, 100000] = 1.0
    check(big, z.repeat(groups, 1), scores_of(657, groups, 2), 16)


@pytest.mark.parametrize("at", [0, 9000, BIG.vocab - 1])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("nan")])
def test_rows_that_are_not_finite(big, bad, at):
    groups = large_call(3)
    z = normal(658, 3 * groups, BIG)
    z[2, at] = bad                                                  # group 0; the others keep their rankings
    check(big, z, scores_of(659, groups, 3), 4, status=tfl.TFL_E_NONFINITE)
    s = scores_of(660, groups, 3)
    s[0, 2] = float("-inf")
    check(big, z, s, 4)
    done = torch.zeros(groups, 3, dtype=torch.int32, device="cuda")
    done[0, 2] = 1
    check(big, z, scores_of(661, groups, 3), 4, done=done, eos=3)


def test_scores_that_are_not_finite(big):
    groups = large_call(2)
    for bad in (float("nan"), float("inf")):
        s = scores_of(662, groups, 2)
        s[1, 1] = bad
        check(big, normal(663, 2 * groups, BIG), s, 3, status=tfl.TFL_E_NONFINITE)
    s = torch.full((groups, 2), float("-inf"), device="cuda")
    s[1, 1] = -4.0
    check(big, normal(664, 2 * groups, BIG), s, 6)


@pytest.mark.parametrize("eos", [0, BIG.vocab - 1])
def test_ended_beams_and_outputs_in_place(big, eos):
    groups = large_call(4)
    z = normal(665, 4 * groups, BIG)
    z[:, eos] += 9.0
    done = torch.zeros(groups, 4, dtype=torch.int32, device="cuda")
    done[0, 1] = done[0, 3] = done[1] = 1
    s = scores_of(666, groups, 4)
    s[0, 1] = -0.5
    check(big, z, s, 8, done=done, eos=eos)
    ref = check(big, z, s, 4, done=done, eos=eos)
    out = outputs(groups, 4, True) | {"out_scores": s, "out_done": done}
    tfl.tfl_beam_select(big, z, s, eos=eos, done=done, **out)
    assert all(torch.equal(out[k], ref[k]) for k in ref)


@pytest.mark.parametrize("below", [0.5, 4.0, 9.0, 13.25, 14.0])
def test_sums_of_equal_logits(big, below):
    V, groups = BIG.vocab, large_call(2)
    z = torch.full((2, V), 2.0 - below, dtype=torch.bfloat16, device="cuda")
    z[0, V // 3], z[1, V - 1] = 2.0, 2.0
    out = outputs(groups, 2)
    tfl.tfl_beam_select(big, z.repeat(groups, 1), torch.zeros(groups, 2, device="cuda"), **out)
    assert big.status() == tfl.TFL_OK
    ref = -np.log1p((V - 1) * np.exp(-below))
    got = out["out_scores"].double().cpu().numpy()
    assert all(sorted(ids) == [V // 3, V - 1] for ids in out["ids"].tolist())
    assert (np.abs(got - ref) <= 2.0 ** -24 * abs(ref) + 2.0 ** -28).all(), got - ref
