"""The shared attention's wait probe at its border: a loader told to stop at a block that some CTA has ends in TFL_E_DEVICE, one that
is told to stop past every CTA's last block never stops, and the call is as ever."""
import pytest
import torch

from gqa_decoder_forward_gb300 import tfl
from tests.test_gpu_shared_attn import Case
from tests.test_gpu_shared_waits import runners  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,prefix,streams,tails,blocks", [     # blocks: of the CTA that has most, on 152 SMs
    ("tiny", [65], [3], [2, 2, 2], 1),
    ("33b", [20000], [16], [100] * 16, 11),
    ("33b", [9000, 3000], [5, 2], [600, 1, 1, 1, 300, 40, 0], 8)])
@pytest.mark.parametrize("past", [-2, -1, 0, 1, 2, 5, 13, 1000])
def test_a_loader_stops_where_a_block_is(runners, name, prefix, streams, tails, blocks, past):  # noqa: F811
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("the units are dealt out to 152 SMs")
    r = runners[name]
    c = Case(r, prefix, streams, tails, seed=510)
    before = c.run()
    out = torch.full_like(c.q, 7.0)
    tfl.tfl_shared_wait_probe(r, c.batch, 0, c.q, out, 2 * blocks + past, 10000)
    status = tfl.tfl_status(r.model)
    if past < 0:
        assert status == tfl.TFL_E_DEVICE
    else:
        assert status == tfl.TFL_OK and torch.equal(out, before)
    assert tfl.tfl_status(r.model) == tfl.TFL_OK and torch.equal(c.run(), before)
