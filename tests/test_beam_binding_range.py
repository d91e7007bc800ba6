"""What the binding of the beam operators refuses because the library cannot see it: numbers that do not fit the C ints they
become (ctypes would keep their low halves), batches made for other lengths of their prefixes, and caches on another device than
their model's (no GPU: devices are stand-ins)."""
import types

import pytest
import torch

from tests.test_beam_binding import GOOD, HEADS, VOCAB, cache, model, null_refused, runner, t
from gqa_decoder_forward_gb300 import build, synth, tfl


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def test_first_row_of_a_reordering():
    batch = tfl.KVRows([cache(), cache()], [0, 1], [2, 3])
    for first in (2 ** 32, 2 ** 31, -2 ** 31 - 1):
        with pytest.raises(ValueError):
            tfl.tfl_kv_reorder_rows(model(), batch, first, t(2), stream=0)
    null_refused(tfl.tfl_kv_reorder_rows, model(), batch, 16, t(2))


def test_a_step_takes_the_prefixes_its_batch_was_made_for():
    ids, logits = t(2), t(2, VOCAB, dtype=torch.bfloat16)
    go = lambda batch: tfl.tfl_decode_step_shared(runner(), batch, ids, logits, stream=0)  # noqa: E731
    for n_prefix in (6, 8, 0):                                   # positions that the step would not keep to
        with pytest.raises(ValueError):
            go(tfl.SharedRows([cache(7)], [2], [cache(), cache()], [n_prefix]))
    with pytest.raises(ValueError):
        go(tfl.SharedRows([None, cache(7)], [1, 1], [cache(), cache()], [0, 6]))
    prefix = cache(7)
    grown = tfl.SharedRows([prefix, None], [1, 1], [cache(), cache()])
    null_refused(tfl.tfl_decode_step_shared, runner(), grown, ids, logits)
    prefix.length = 8                                            # after the tails were made
    with pytest.raises(ValueError):
        go(grown)
    null_refused(tfl.tfl_decode_step_shared, runner(), tfl.SharedRows([cache(7)], [2], [cache(), cache()], [7]), ids, logits)


@pytest.mark.parametrize("big", [2 ** 32 + 2, 2 ** 31, -2 ** 31 - 1])
def test_single_numbers(big):
    with pytest.raises(ValueError):
        tfl.tfl_beam_select(model(), **GOOD, eos=big, stream=0)
    batch, q = tfl.SharedRows([cache(7)], [1], [cache()], pos=[7]), t(1, HEADS * 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tfl.tfl_shared_attention(runner(), batch, big, q, q, stream=0)
    for lose, limit in ((big, 1), (0, big)):
        with pytest.raises(ValueError):
            tfl.tfl_shared_wait_probe(runner(), batch, 0, q, q, lose, limit, stream=0)


@pytest.mark.parametrize("model_on,current,buffer_on", [(0, 1, 1), (0, 1, 0), (0, 0, 1), (1, 0, 0), (0, 1, None)])
def test_caches_are_made_on_their_models_device(monkeypatch, model_on, current, buffer_on):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    m = types.SimpleNamespace(handle=None, cfg=tfl.config(synth.TINY), workspace=types.SimpleNamespace(get_device=lambda: model_on))
    buffer = None if buffer_on is None else types.SimpleNamespace(
        is_cuda=True, is_contiguous=lambda: True, get_device=lambda: buffer_on, stride=lambda: (1,), device=f"cuda:{buffer_on}")
    with pytest.raises(ValueError):
        tfl.KV(m, 100, buffer=buffer)


def test_a_runners_workspace_lies_on_its_models_device():
    assert tfl.SharedRunner(model()).workspace.device == model().workspace.device
