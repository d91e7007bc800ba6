"""Numbers that the binding of the beam operators hands to the library as C ints: refused where they do not fit, since ctypes
would keep their low halves (no GPU)."""
import pytest

from tests.test_beam_binding import cache, model, null_refused, t
from gqa_decoder_forward_gb300 import build, tfl


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def test_first_row_of_a_reordering():
    batch = tfl.KVRows([cache(), cache()], [0, 1], [2, 3])
    for first in (2 ** 32, 2 ** 31, -2 ** 31 - 1):
        with pytest.raises(ValueError):
            tfl.tfl_kv_reorder_rows(model(), batch, first, t(2), stream=0)
    with pytest.raises(TypeError):
        tfl.tfl_kv_reorder_rows(model(), batch, 1.0, t(2), stream=0)
    null_refused(tfl.tfl_kv_reorder_rows, model(), batch, 16, t(2))
