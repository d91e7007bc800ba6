"""Attention over the longest 4-bit caches: joins whose groups pass 48 KB of shared memory, up to as many units as
a full grid has warps."""
import numpy as np
import pytest
import torch

from gqa_decoder_forward_gb300 import tfl
from tests import kv4_ref as ref
from tests.test_gpu_kv4 import _built, attend, check, cuda_bf16, filled, queries, rows_like_keys, values64  # noqa: F401

pytestmark = pytest.mark.gpu


def test_one_head_over_230000_keys():
    n = 230000                                                      # 7,188 steps in units of 8: 113 groups
    kv, kq, vq = filled(500, 1, n, n)
    attn = tfl.KV4Attention(4, 1, max_rows=3, max_positions=n)
    q = queries(501, 3, 4, 0.4)
    window = attend(attn, [kv], [n - 3], [3], q)
    check(window[[0, 2]], q[[0, 2]], [n - 3, n - 1], kq, vq)
    for i in range(3):
        assert (attend(attn, [kv], [n - 3 + i], [1], q[i: i + 1])[0] == window[i]).all()


@pytest.mark.parametrize("n_kv,g", [(1, 8), (2, 3)])
def test_the_last_of_2_to_the_20_positions(n_kv, g):
    """All but the first and the last 40 positions hold zeros: keys that score 0 and stand for 0."""
    cap, m = 1 << 20, 40
    kv = tfl.KV4(1, n_kv, cap)
    kv.buffer[(cap // 128 * 4 + 255) // 256 * 256:].zero_()
    at = [0, cap - m]
    x = [(rows_like_keys(510 + i, m, n_kv), rows_like_keys(520 + i, m, n_kv)) for i in range(2)]
    for p, (k, v) in zip(at, x):
        tfl.tfl_kv4_write(tfl.KV4Rows([kv], [p], [m]), 0, cuda_bf16(k), cuda_bf16(v))
    attn = tfl.KV4Attention(n_kv * g, n_kv, max_rows=1, max_positions=cap)
    q = queries(530, 1, n_kv * g)
    got = attend(attn, [kv], [cap - 1], [1], q)
    kq, vq = (np.concatenate([values64(a[i]) for a in x]) for i in range(2))
    top = max(np.abs(a[1]).max() for a in x)
    for j in range(n_kv * g):
        s = kq[:, j // g] @ q[0, j].astype(np.float64) / np.sqrt(128)
        high = max(s.max(), 0.0)
        p = np.exp(s - high)
        p /= p.sum() + (cap - 2 * m) * np.exp(-high)
        want = p @ vq[:, j // g]
        # the restatement's bound with the zeros left out (they add nothing): 2^-8 |out|, then 2^-11 and less of
        # sum P (|z| + s n), where |z| + s n <= 3 max |v|; doubled
        tol = 2.0 ** -7 * np.abs(want) + 2.0 ** -10 * p.sum() * 3 * top
        assert (np.abs(got[0, j] - want) <= tol).all(), j
