"""tfl_beam_select where chunks of a row lie far below its largest logit: a vocabulary mask that adds a large negative
number to a run of ids leaves the row's sum what it is without them.  The tolerance is test_gpu_beam_select's."""
import pytest
import torch

from gqa_decoder_forward_gb300 import build
from tests.test_gpu_beam_select import BIG, check, normal, plain_model, scores_of

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
