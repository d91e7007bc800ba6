"""The attention's bounded wait for keys, made to run out on purpose with no fault: a step is announced and
never copied.  The warp gives up, its copies in flight end, the status says so, and the next call is as ever."""
import pytest
import torch

from gqa_decoder_forward_gb300 import tfl
from tests.test_gpu_kv4 import _built, attend, cuda_bf16, filled, queries  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_kv,pos0,rows", [(1, 30, 1),      # one step
                                            (1, 40, 1),      # two: both stages hold one
                                            (8, 4000, 2),    # units of four steps, one to a warp
                                            (8, 20000, 16)])  # units one after the other
@pytest.mark.parametrize("lose", [0, 1, 2, 5])
def test_a_step_that_never_comes_ends_in_the_status_word(n_kv, pos0, rows, lose):
    n = pos0 + rows
    kv, _, _ = filled(400, n_kv, n, n)
    attn = tfl.KV4Attention(7 * n_kv, n_kv, max_rows=rows, max_positions=n)
    q = queries(401, rows, 7 * n_kv)
    before = attend(attn, [kv], [pos0], [rows], q)
    tq = cuda_bf16(q).view(rows, -1)
    out = torch.zeros_like(tq)
    tfl.tfl_kv4_wait_probe(attn, tfl.KV4Rows([kv], [pos0], [rows]), 0, tq, out, lose, 10000)
    steps = 1 if pos0 == 30 else 2 if pos0 == 40 else 4 if pos0 == 4000 else 6   # that some warp has, at least
    if lose < steps:
        with pytest.raises(tfl.TflError) as e:
            tfl._check(tfl.tfl_kv4_attn_status(attn))
        assert e.value.code == tfl.TFL_E_DEVICE
    assert tfl.tfl_kv4_attn_status(attn) == tfl.TFL_OK            # read and cleared, or never raised
    assert (attend(attn, [kv], [pos0], [rows], q) == before).all()


def test_probe_arguments_are_checked():
    kv, _, _ = filled(410, 1, 10, 10)
    attn = tfl.KV4Attention(8, 1, max_rows=1, max_positions=10)
    q = torch.zeros((1, 1024), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    for lose, limit in ((-1, 100), (0, 0), (0, (1 << 20) + 1)):
        with pytest.raises(tfl.TflError) as e:
            tfl.tfl_kv4_wait_probe(attn, tfl.KV4Rows([kv], [9], [1]), 0, q, out, lose, limit)
        assert e.value.code == tfl.TFL_E_ARG
