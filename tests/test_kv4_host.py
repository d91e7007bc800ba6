"""The 4-bit cache without a GPU: sizes, refusals, and the numpy restatement that the
GPU tests compare with."""
import ctypes

import numpy as np
import pytest

from gqa_decoder_forward_gb300 import build, tfl
from tests import kv4_ref as ref


@pytest.fixture(scope="module")
def L():
    build.build()
    return tfl.lib()


def test_bytes_are_the_tables_and_the_tiles(L):
    assert tfl.tfl_kv4_bytes(1, 1, 1) == 256 + ref.TILE
    assert tfl.tfl_kv4_bytes(52, 8, 131072) == 4096 + 52 * 1024 * 8 * ref.TILE
    assert tfl.tfl_kv4_bytes(3, 5, 129) == 256 + 3 * 2 * 5 * ref.TILE
    # 144 bytes a position and head: 3.56 times less than two bf16 rows of 128
    assert ref.TILE == 128 * 144 and 512 / 144 > 3.5
    # sizes whose products pass 32 bits
    assert tfl.tfl_kv4_bytes(1024, 64, 1 << 20) == (1 << 15) + 1024 * 8192 * 64 * ref.TILE


@pytest.mark.parametrize("sizes", [(0, 8, 128), (1025, 8, 128), (1, 0, 128), (1, 65, 128), (1, 8, 0),
                                   (1, 8, (1 << 20) + 1), (-1, 8, 128), (1, -8, 128), (1, 8, -128)])
def test_cache_sizes_outside_the_range_are_refused(L, sizes):
    assert tfl.tfl_kv4_bytes(*sizes) == 0
    h = ctypes.c_void_p(1)
    assert L.tfl_kv4_alloc(sizes[0], sizes[1], 128, sizes[2], 256, 1 << 40, ctypes.byref(h)) == tfl.TFL_E_ARG
    assert not h.value and b"refused" in L.tfl_last_error()


def test_other_head_sizes_are_refused(L):
    assert L.tfl_kv4_bytes(1, 8, 64, 128) == 0
    assert L.tfl_kv4_attn_bytes(56, 8, 64, 1, 128) == 0


def test_alloc_refuses_buffers_that_do_not_fit(L):
    h = ctypes.c_void_p()
    n = tfl.tfl_kv4_bytes(1, 8, 128)
    for buf, size, code in ((None, n, tfl.TFL_E_ARG), (8, n, tfl.TFL_E_ARG), (256, n - 1, tfl.TFL_E_WORKSPACE)):
        assert L.tfl_kv4_alloc(1, 8, 128, 128, buf, size, ctypes.byref(h)) == code
    assert L.tfl_kv4_alloc(1, 8, 128, 128, 256, n, None) == tfl.TFL_E_ARG


@pytest.mark.parametrize("n_q,n_kv,rows,pos", [(7, 2, 1, 128), (17, 1, 1, 128), (4, 8, 1, 128), (0, 1, 1, 128),
                                               (8, 1, 0, 128), (8, 1, 65, 128), (8, 1, 1, 0), (130, 65, 1, 128),
                                               (8, 1, 1, (1 << 20) + 1)])
def test_attention_sizes_outside_the_range_are_refused(L, n_q, n_kv, rows, pos):
    assert L.tfl_kv4_attn_bytes(n_q, n_kv, 128, rows, pos) == 0
    h = ctypes.c_void_p(1)
    assert L.tfl_kv4_attn_init(n_q, n_kv, 128, rows, pos, 256, 1 << 40, ctypes.byref(h)) == tfl.TFL_E_ARG
    assert not h.value


def test_attention_workspace_is_checked(L):
    h = ctypes.c_void_p()
    n = L.tfl_kv4_attn_bytes(56, 8, 128, 16, 4096)
    assert n > 0
    for ws, size, code in ((None, n, tfl.TFL_E_ARG), (128, n, tfl.TFL_E_ARG), (256, n - 1, tfl.TFL_E_WORKSPACE)):
        assert L.tfl_kv4_attn_init(56, 8, 128, 16, 4096, ws, size, ctypes.byref(h)) == code


def test_null_objects_are_refused(L):
    one, kvs = (ctypes.c_int * 1)(1), (ctypes.c_void_p * 1)(None)
    for arr, p, r in ((None, one, one), (kvs, None, one), (kvs, one, None), (kvs, one, one)):
        assert L.tfl_kv4_write(arr, 1, 0, p, r, 256, 512, 128, None) == tfl.TFL_E_ARG
        assert L.tfl_kv4_read(arr, 1, 0, p, r, 256, 512, 128, None) == tfl.TFL_E_ARG
    assert L.tfl_kv4_write(kvs, 17, 0, one, one, 256, 512, 128, None) == tfl.TFL_E_ARG
    assert L.tfl_kv4_write(kvs, 0, 0, one, one, 256, 512, 128, None) == tfl.TFL_E_ARG
    assert L.tfl_kv4_attention(None, kvs, 1, 0, one, one, 256, 1024, 512, 1024, None) == tfl.TFL_E_ARG
    assert L.tfl_kv4_attn_status(None, None) == tfl.TFL_E_ARG
    assert L.tfl_kv4_reset(None, 0) == tfl.TFL_E_ARG
    assert L.tfl_kv4_length(None) == -1 and L.tfl_kv4_capacity(None) == -1
    L.tfl_kv4_free(None)
    L.tfl_kv4_attn_free(None)


# ---- the restatement ------------------------------------------------------------------

def _rows(seed, n, n_kv=2):
    r = np.random.default_rng(seed)
    x = r.normal(size=(n, n_kv, 128)) * np.exp(r.normal(size=128))
    return ref.from_bits(ref.bf16_bits(x.astype(np.float32)))


def test_a_group_stands_for_its_numbers_within_half_a_scale():
    x = _rows(1, 200)
    code, scale, zero = ref.quantise(x)
    s = np.repeat(scale, ref.GROUP, -1).astype(np.float64)
    assert (np.abs(ref.values(code, scale, zero) - x) <= s * (0.5 + 15 * 2.0 ** -8) + 1e-30).all()
    assert code.max() == 15 and code.min() == 0


def test_groups_of_one_number_and_groups_that_are_not_finite():
    x = np.zeros((4, 1, 128), np.float32)
    x[0] = 3.25
    x[1, 0, 5], x[1, 0, 70] = np.inf, np.nan
    x[2, 0, 0], x[2, 0, 1] = 3e38, -3e38      # max - min overflows
    x[3, 0, :64] = np.float32(2.0) ** -133 * np.arange(64)  # subnormal numbers
    code, scale, zero = ref.quantise(x)
    v = ref.values(code, scale, zero)
    assert (v[0] == 3.25).all() and np.isnan(v[1]).all()
    assert np.isnan(v[2, 0, :64]).all() and (v[2, 0, 64:] == 0).all()
    assert np.isfinite(v[3]).all()


def test_layout_round_trip_through_a_permuted_table():
    c = ref.Cache(2, 3, 300, fill=0xEE, table=[2, 0, 1])
    r = np.random.default_rng(2)
    n = 300
    code = r.integers(0, 16, (2, n, 3, 128), dtype=np.uint8)
    scale = ref.from_bits(ref.bf16_bits(r.random((2, n, 3, 2)).astype(np.float32)))
    zero = ref.from_bits(ref.bf16_bits(r.normal(size=(2, n, 3, 2)).astype(np.float32)))
    for kind in range(2):
        for p in range(n):
            c.put(1, p, kind, code[kind, p], scale[kind, p], zero[kind, p])
    for kind in range(2):
        a, s, z = c.get(1, n, kind)
        assert (a == code[kind]).all() and (s == scale[kind]).all() and (z == zero[kind]).all()
    assert (c.bytes[c.table_bytes: c.table_bytes + 3 * 3 * ref.TILE] == 0xEE).all()   # layer 0 untouched


def test_attention_reference_is_the_softmax_average():
    x = _rows(3, 20, 1)
    kq, vq = ref.quantise(x), ref.quantise(_rows(4, 20, 1))
    q = np.zeros((2, 128))
    out, bound = ref.attention(q, 9, kq, vq)
    assert np.allclose(out, ref.values(*vq)[:10, 0].mean(0))
    # 2^-8 |out| and 2^-11 sum P s n are each below 2^-8 of the largest |z| + s n, the rest far below
    top = (np.abs(np.repeat(vq[2], 64, -1)) + ref.values(vq[0], vq[1], 0 * vq[2])).max()
    assert (bound > 0).all() and (bound < 2.0 ** -7 * top).all()
