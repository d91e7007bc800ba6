"""Attention over the 4-bit cache where the scales of values, and the scores, lie far apart: the
operand scales that the kernel keeps per column, against the 64-bit restatement and its bound."""
import numpy as np
import pytest

from gqa_decoder_forward_gb300 import tfl
from tests import kv4_ref as ref
from tests.test_gpu_kv4 import _built, attend, check, cuda_bf16, make, queries, rows_like_keys  # noqa: F401

pytestmark = pytest.mark.gpu


def bf16(x):
    return ref.from_bits(ref.bf16_bits(np.asarray(x, np.float32)))


def cache_of(k, v):
    """A library cache of rows k, v [n, n_kv, 128], what is never written reading as NaN."""
    _, kv = make(1, k.shape[1], k.shape[0], 0xFF)
    tfl.tfl_kv4_write(tfl.KV4Rows([kv], [0], [k.shape[0]]), 0, cuda_bf16(k), cuda_bf16(v))
    return kv


@pytest.mark.parametrize("n", [128, 700])
@pytest.mark.parametrize("up", [24, 30, 40])
def test_large_values_of_low_scores_before_ordinary_values_of_high_ones(n, up):
    """The first 32 keys of every 128 have values 2^up times the others' and, in some columns, scores some 60
    (log2) below theirs: they set a unit's operand scale and then weigh nothing."""
    k, v = rows_like_keys(200, n, 1), rows_like_keys(201, n, 1)
    first = np.arange(n) % 128 < 32
    v[first] *= np.float32(2.0 ** up)
    k[:, 0, 0] = np.where(first, -30.0, 0.0)
    kv = cache_of(k, v)
    q = queries(202, 1, 8)
    q[0, :, 0] = [16, 17, -16, 0, 8, 4, 30, 2]   # 0.1275 x 30 x 16 = 61
    attn = tfl.KV4Attention(8, 1, max_rows=1, max_positions=n)
    check(attend(attn, [kv], [n - 1], [1], q), q, [n - 1], ref.quantise(k), ref.quantise(v))


@pytest.mark.parametrize("n", [40, 700])
@pytest.mark.parametrize("a,b", [(30, 0), (0, 40), (60, -60), (-50, 50), (None, None)])
def test_the_halves_of_a_value_do_not_share_an_operand_scale(a, b, n):
    """Values whose dims 0..63 and 64..127 differ by up to 2^120 (None: one way and the other, by 32 positions)."""
    k, v = rows_like_keys(210, n, 1), rows_like_keys(211, n, 1)
    if a is None:
        turn = (np.arange(n) // 32 % 2 * 60 - 30)[:, None]
        v[:, 0, :64] *= (2.0 ** turn).astype(np.float32)
        v[:, 0, 64:] *= (2.0 ** -turn).astype(np.float32)
    else:
        v[..., :64] *= np.float32(2.0 ** a)
        v[..., 64:] *= np.float32(2.0 ** b)
    kv = cache_of(k, v)
    q = queries(212, 3, 8)
    attn = tfl.KV4Attention(8, 1, max_rows=3, max_positions=n)
    check(attend(attn, [kv], [n - 3], [3], q), q, range(n - 3, n), ref.quantise(k), ref.quantise(v))


def test_a_rows_bits_next_to_the_threshold_do_not_depend_on_its_neighbour():
    """One row's largest weight lies just above 2^15 in operand units, where rounding to fp16 takes it to 2^15, in a step
    in which the row beside it moves its maximum.  What follows is 2^29 smaller, in dims where all else is 0."""
    n = 97
    k, v = np.zeros((n, 1, 128)), np.zeros((n, 1, 128))
    v[:32, 0, 0] = 15                                   # scale 1, first: operand scale 2^6
    k[32, 0, 0] = 15 * 2.0 ** -4                        # scale 2^-4
    v[32, 0, 0] = 15 * 2.0 ** 9                         # scale 2^9, weight 2^(0.1275 x 15 x 2^-12) = 1.00032
    r = np.random.default_rng(220)
    v[64:96, 0, 1:64] = 2.0 ** -20 * r.uniform(0, 25, (32, 63))
    q = np.zeros((2, 1, 128), np.float32)
    q[0, 0, 0], q[1, 0, 0] = 2.0 ** -8, 100             # the neighbour's score at key 32: 12 above those before
    k, v = bf16(k), bf16(v)
    kv = cache_of(k, v)
    attn = tfl.KV4Attention(1, 1, max_rows=2, max_positions=n)
    alone = attend(attn, [kv], [95], [1], q[:1])
    window = attend(attn, [kv], [95], [2], q)
    assert (window[0] == alone[0]).all()
    kq, vq = ref.quantise(k), ref.quantise(v)
    out, bound = ref.attention(q[0].astype(np.float64), 95, kq, vq)
    # An odd dim's codes are the high halves of bytes: their sum is a sixteenth of the difference of the bytes' sum and the
    # low codes'.  Both are fp32 sums in chains of at most 64 steps (the restatement's 2^-17 each), so the dim below it,
    # which alone is large here, adds 2 x 2^-17 / 16 = 2^-20 of its own sum.
    low, _ = ref.attention(q[0].astype(np.float64), 95, kq, (vq[0], vq[1], 0 * vq[2]))
    bound[:, 1::2] += 2.0 ** -20 * low[:, 0::2]
    assert (np.abs(alone[0] - out) <= bound).all()


@pytest.mark.parametrize("rise,fall", [(12, 12), (12, 4), (9, 16), (20, 12), (12, -4), (-12, -4), (3, 12)])  # values to 2^90
def test_scores_that_rise_while_the_values_scales_fall(rise, fall):
    """Units of eleven steps (64 heads, of which two differ), each step's scores 2^rise above the one before (in the first row's
    weights) and its values 2^fall below: the maximum moves again and again, and what came before counts, or not, or
    counts alone."""
    n, n_kv = 8600, 64                                  # 269 steps over 28 units at most: ten or more to a unit
    steps = -(-(-(-n // 32)) // 28)
    at = np.arange(n) // 32 % steps
    r = np.random.default_rng(230)
    k, v = 0.1 * r.normal(size=(n, 2, 128)), r.normal(size=(n, 2, 128))
    k[:, 0, 0] = k[:, 1, 0] = rise * at                 # 0.1275 x 8 = 1.02 in the scores' log2
    v *= 2.0 ** (50 - fall * at)[:, None, None]
    k, v = bf16(k), bf16(v)
    kv = cache_of(np.tile(k, (1, n_kv // 2, 1)), np.tile(v, (1, n_kv // 2, 1)))
    q = queries(231, 1, n_kv, 0.3)
    q[0, :, 0] = np.resize([8, 8, 4, -8, 0, 9], n_kv)
    attn = tfl.KV4Attention(n_kv, n_kv, max_rows=1, max_positions=n)
    got = attend(attn, [kv], [n - 1], [1], q)
    kq, vq = ref.quantise(k), ref.quantise(v)
    for h in range(0, 12, 2):                           # heads h and h + 1 hold the two that differ
        check(got[:, h: h + 2], q[:, h: h + 2], [n - 1], kq, vq, f"heads {h}, {h + 1}")
