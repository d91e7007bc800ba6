"""What the binding of the 4-bit cache checks before it calls the library (no GPU)."""
import types

import pytest
import torch

from gqa_decoder_forward_gb300 import build, tfl


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


VOCAB = 40


def runner():
    """Stands for a KV4Runner without a model: the library refuses its NULL handles."""
    null = types.SimpleNamespace(handle=None, shape=types.SimpleNamespace(vocab=VOCAB))
    ws = torch.empty(0, dtype=torch.uint8)
    return types.SimpleNamespace(model=null, attention=null, step_ws=ws, prompt_ws=ws)


def caches(n):
    return [types.SimpleNamespace(handle=None)] * n


def ids(n, dtype=torch.int32):
    return torch.zeros(n, dtype=dtype)


def logits(n, dtype=torch.bfloat16):
    return torch.zeros(n, VOCAB, dtype=dtype)


@pytest.mark.parametrize("kvs,i,rows,out", [
    (2, ids(2), [1], logits(2)),                       # the row counts end before the caches
    (1, ids(2), [1, 1], logits(2)),
    (2, ids(4), [2, 3], logits(5)),                    # fewer ids than rows
    (2, ids(5), [2, 3], logits(4)),                    # fewer rows of logits
    (1, ids(1, torch.int64), [1], logits(1)),
    (1, ids(1), [1], logits(1, torch.float32)),
])
def test_a_step_checks_the_lengths_of_its_arrays(kvs, i, rows, out):
    with pytest.raises(ValueError):
        tfl.tfl_decode_step_kv4(runner(), caches(kvs), i, rows, out, stream=0)


@pytest.mark.parametrize("i,out,all_rows", [(ids(3), logits(2), True), (ids(3), logits(0), False), (ids(0), None, False),
                                            (ids(3, torch.int64), None, False), (ids(3), logits(3, torch.float32), True)])
def test_a_prompt_chunk_checks_its_ids_and_logits(i, out, all_rows):
    with pytest.raises(ValueError):
        tfl.tfl_prefill_chunk_kv4(runner(), caches(1)[0], i, out, all_rows, stream=0)


def test_lengths_that_fit_reach_the_library():
    for call, args in ((tfl.tfl_decode_step_kv4, (caches(2), ids(6), [2, 3], logits(5))),
                       (tfl.tfl_prefill_chunk_kv4, (caches(1)[0], ids(3), logits(1), False))):
        with pytest.raises(tfl.TflError) as e:
            call(runner(), *args, stream=0)
        assert e.value.code == tfl.TFL_E_ARG


def test_a_cache_takes_memory_of_the_current_device_alone():
    n = tfl.tfl_kv4_bytes(1, 1, 128)
    with pytest.raises(ValueError):
        tfl.KV4(1, 1, 128, buffer=torch.empty(n, dtype=torch.uint8))     # the host's
    with pytest.raises(ValueError):
        tfl.KV4(1, 1, 128, buffer=torch.empty(2 * n, dtype=torch.uint8)[::2])


def rows_on(device, heads=2, rows=3):
    """Stands for a bf16 CUDA tensor [rows, heads, 128] of a device."""
    return types.SimpleNamespace(dtype=torch.bfloat16, is_cuda=True, shape=(rows, heads, 128),
                                 stride=lambda: (heads * 128, 128, 1), get_device=lambda: device, data_ptr=lambda: 256)


def cache_on(device, n_kv=2):
    return types.SimpleNamespace(handle=None, n_kv=n_kv, buffer=types.SimpleNamespace(get_device=lambda: device))


def test_rows_of_another_device_than_the_caches_are_refused():
    batch = tfl.KV4Rows([cache_on(0)], [0], [3])
    attn = types.SimpleNamespace(handle=None, n_q=2)
    here, there = rows_on(0), rows_on(1)
    for call in (tfl.tfl_kv4_write, tfl.tfl_kv4_read):
        for k, v in ((here, there), (there, here), (there, there)):
            with pytest.raises(ValueError):
                call(batch, 0, k, v, stream=0)
        with pytest.raises(tfl.TflError):                                # the library, of the NULL cache
            call(batch, 0, here, here, stream=0)
    for q, out in ((here, there), (there, here)):
        with pytest.raises(ValueError):
            tfl.tfl_kv4_attention(attn, batch, 0, q, out, stream=0)


def test_ids_or_logits_of_another_device_are_refused():
    r = runner()
    r.step_ws = types.SimpleNamespace(get_device=lambda: 0, device="cuda:0")
    with pytest.raises(ValueError):
        tfl.tfl_decode_step_kv4(r, caches(1), ids(1), [1], logits(1), stream=0)
    with pytest.raises(ValueError):
        tfl.tfl_prefill_chunk_kv4(r, caches(1)[0], ids(1), logits(1), False, stream=0)


@pytest.mark.parametrize("pos0,rows", [([2 ** 32 + 3], [1]), ([3], [2 ** 32 + 1]), ([-2 ** 31 - 1], [1]), ([5.0], [1]), ([5], [1.0])])
def test_positions_and_rows_that_no_int_holds_are_refused_and_change_nothing(pos0, rows):
    with pytest.raises((ValueError, TypeError)):
        tfl.KV4Rows([cache_on(0)], pos0, rows)
    batch = tfl.KV4Rows([cache_on(0)], [1], [2])
    with pytest.raises((ValueError, TypeError)):
        batch.set(pos0, rows)
    assert (list(batch.pos0), list(batch.rows), batch.total) == ([1], [2], 2)


def test_one_row_may_be_a_tensor_of_one_row_beside_a_part_of_wider_rows():
    one, wide = rows_on(0, rows=1), rows_on(0, rows=5)
    wide.stride = lambda: (5 * 256, 128, 1)
    with pytest.raises(tfl.TflError):                                    # the library, of the NULL cache
        tfl.tfl_kv4_write(tfl.KV4Rows([cache_on(0)], [0], [1]), 0, one, wide, stream=0)
    with pytest.raises(ValueError):
        tfl.tfl_kv4_write(tfl.KV4Rows([cache_on(0)], [0], [2]), 0, rows_on(0), wide, stream=0)


def test_a_call_without_rows_takes_an_empty_tensor_of_any_strides():
    none = rows_on(0, rows=0)
    none.stride = lambda: (0, 0, 0)
    for call in (tfl.tfl_kv4_write, tfl.tfl_kv4_read):
        with pytest.raises(tfl.TflError):                                # the library, of the NULL cache
            call(tfl.KV4Rows([cache_on(0)], [0], [0]), 0, none, none, stream=0)
        with pytest.raises(ValueError):
            call(tfl.KV4Rows([cache_on(0)], [0], [1]), 0, none, none, stream=0)
