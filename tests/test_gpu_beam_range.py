"""tfl_beam_select over fp32's whole range.  Chunks of a row far below its largest logit: a vocabulary mask that adds a large negative
number to a run of ids leaves the row's sum what it is without them.  Scores below fp32's lowest number: compared in 64 bits
all the same.  The tolerance is test_gpu_beam_select's."""
import numpy as np
import pytest
import torch

from gqa_decoder_forward_gb300 import build, tfl
from tests import beam_ref
from tests.test_gpu_beam_select import BIG, TINY, check, normal, outputs, plain_model, scores_of

pytestmark = pytest.mark.gpu
CHUNK = 8192   # logits of a row that are summed together


@pytest.fixture(scope="module")
def big():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    build.build()
    return plain_model(BIG, 64)


FAR = [-200.0, -16320.0, -16384.0, -32768.0, -2.0 ** 17, -2.5e5, -2.8e5, -3e5, -3.5e5, -4e5, -5e5, -5.5e5, -7.9e5, -1e6, -1e9,
       float(torch.finfo(torch.bfloat16).min)]


@pytest.mark.parametrize("groups", [1, 4])        # a CTA per chunk on SMs of their own, and several to an SM
@pytest.mark.parametrize("low", FAR)
def test_chunks_far_below_the_largest_logit(big, low, groups):
    z = normal(600, 4, BIG)
    z[0, CHUNK: 2 * CHUNK] = low                  # one whole chunk
    z[1, CHUNK // 2: 5 * CHUNK + 7] = low         # some, and parts of others
    z[1, 3 * CHUNK + 5] = 10.0                    # an ordinary logit among them
    z[2, 100:] = low                              # all but a few ids of the first chunk
    z[3, : 20 * CHUNK] = low                      # all but the last, partial chunk
    check(big, z.repeat(groups, 1), scores_of(601, groups, 4), 32)


@pytest.mark.parametrize("top", [10.0, 3.5, -7.0, 120.0])
def test_chunks_that_are_all_one_far_number(big, top):
    """A number of its own for each row, from -2^17 to -2^20 in steps of one to four bf16 numbers."""
    patterns = torch.arange(0xC800, 0xC980, 6, dtype=torch.int32)
    low = ((patterns - 65536) << 16).view(torch.float32)
    assert len(low) == 64 and low[0] == -2.0 ** 17 and low[-1] > -2.0 ** 20
    z = normal(602, 64, BIG)
    z[:, 77] = top + 100.0 if top < 0 else top
    z[:, 2 * CHUNK: 3 * CHUNK] = low.to(torch.bfloat16).cuda()[:, None]
    if top < 0:
        z -= 100.0
    check(big, z, scores_of(603, 16, 4), 32)


@pytest.fixture(scope="module")
def models(big):
    return {"tiny": plain_model(TINY, 64), "33b": big}


LOWEST = float(torch.finfo(torch.float32).min)


def rows_beyond(kind, V):
    """[4, V] logits, twelve ids of each row allowed, and [1, 4] scores: many candidates' scores are below fp32's lowest number."""
    gen = torch.Generator().manual_seed(604)
    z = torch.full((4, V), float("-inf"), dtype=torch.float64)
    span = {"logits": 6.7e38, "scores": 3e38, "both": 6.7e38}[kind]       # from the largest down
    scores = {"logits": [-3.0, -2.0, -5.0, -4.0], "scores": [-3.39e38, -3.395e38, LOWEST, -3.38e38],
              "both": [-3.2e38, -1e38, -3.3e38, -2e38]}[kind]
    for b in range(4):
        allowed = torch.randperm(V, generator=gen)[:12]
        z[b, allowed] = 3.35e38 - span * torch.rand(12, generator=gen).double()
        z[b, allowed[0]] = 3.35e38
    return z.to(torch.bfloat16), torch.tensor([scores], dtype=torch.float32)


@pytest.mark.parametrize("n_out", [5, 32])
@pytest.mark.parametrize("kind", ["logits", "scores", "both"])
@pytest.mark.parametrize("name", ["tiny", "33b"])
def test_scores_beyond_fp32(models, name, kind, n_out):
    """Ranked by their 64-bit values all the same; out_scores is -inf where float32 is."""
    m = models[name]
    z, scores = rows_beyond(kind, m.shape.vocab)
    ids, parents, ref, _ = beam_ref.select(z.double().numpy(), scores.double().numpy(), n_out)
    with np.errstate(over="ignore"):
        ref = ref.astype(np.float32)
    assert np.isinf(ref).sum() > 1 or n_out < 32
    assert len(set(parents[0].tolist())) > 1
    out = outputs(1, n_out)
    tfl.tfl_beam_select(m, z.cuda(), scores.cuda(), **out)
    assert m.status() == tfl.TFL_OK
    assert np.array_equal(out["parents"].cpu().numpy(), parents) and np.array_equal(out["ids"].cpu().numpy(), ids)
    got = out["out_scores"].cpu().numpy()
    assert np.array_equal(np.isinf(got), np.isinf(ref))
    fine = np.isfinite(ref)
    assert (np.abs(got[fine].astype(float) - ref[fine]) <= 2.0 ** -23 * np.abs(ref[fine].astype(float)) + 2.0 ** -28).all()
