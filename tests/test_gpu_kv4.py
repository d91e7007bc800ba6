"""The 4-bit cache on the GPU: rows written (the codes of the fp32 formula, bit for bit, and
nothing else touched), read back, and attended, against the numpy restatement in 64 bits."""
import ctypes

import numpy as np
import pytest
import torch

from gqa_decoder_forward_gb300 import synth, tfl
from tests import kv4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gqa_decoder_forward_gb300 import build
    build.build()
    tfl.lib()


def cuda_bf16(x):
    return torch.from_numpy(np.ascontiguousarray(ref.bf16_bits(x)).view(np.int16)).cuda().view(torch.bfloat16)


def host_f32(t):
    return ref.from_bits(t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16))


def rows_like_keys(seed, n, n_kv):
    r = np.random.default_rng(seed)
    x = 1.7 * r.normal(size=(n, n_kv, 128)) * np.exp(0.5 * r.normal(size=(n_kv, 128)))
    return ref.from_bits(ref.bf16_bits(x.astype(np.float32)))


def make(layers, n_kv, cap, fill=0xA5, table=None):
    """A host cache and a library cache over the same bytes (the table rewritten after alloc)."""
    host = ref.Cache(layers, n_kv, cap, fill, table)
    buf = torch.from_numpy(host.bytes.copy()).cuda()
    kv = tfl.KV4(layers, n_kv, cap, buffer=buf)
    if table is not None:
        buf[: host.pages * 4] = torch.from_numpy(host.table.view(np.uint8).copy()).cuda()
    return host, kv


def put_rows(host, layer, pos0, kind, x):
    code, scale, zero = ref.quantise(x)
    for i in range(x.shape[0]):
        host.put(layer, pos0 + i, kind, code[i], scale[i], zero[i])


def same_bytes(host, kv, what=""):
    got = kv.buffer.cpu().numpy()[host.table_bytes:]
    want = host.bytes[host.table_bytes:]
    bad = np.nonzero(got != want)[0]
    assert bad.size == 0, f"{what}: {bad.size} bytes differ, first at {bad[0]}"


# ---- write ------------------------------------------------------------------------------

WRITES = [  # n_kv, capacity, pos0 per stream, rows per stream
    (1, 1, [0], [1]),
    (8, 300, [127], [2]),
    (2, 200, [5], [190]),
    (3, 513, [511], [1]),
    (8, 400, [0, 1, 17, 126, 128, 255, 399], [1, 1, 1, 1, 1, 1, 1]),
    (1, 130, [3, 64, 0, 129], [7, 0, 130, 1]),
    (5, 64, [0] * 16, list(range(16))),
    (4, 1100, [33], [1050]),
]


@pytest.mark.parametrize("n_kv,cap,pos0,rows", WRITES)
@pytest.mark.parametrize("strided", [False, True])
def test_written_codes_are_the_formulas_and_nothing_else_changes(n_kv, cap, pos0, rows, strided):
    pairs = [make(2, n_kv, cap) for _ in pos0]
    n = sum(rows)
    k, v = rows_like_keys(1, n, n_kv), rows_like_keys(2, n, n_kv)
    spare = 2  # rows past the last stream's: not read into any cache
    wide = torch.full((n + spare, 5, n_kv, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    if strided:
        tk, tv = wide[:, 1], wide[:, 3]
    else:
        tk, tv = (torch.full((n + spare, n_kv, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tk[:n], tv[:n] = cuda_bf16(k), cuda_bf16(v)
    tfl.tfl_kv4_write(tfl.KV4Rows([kv for _, kv in pairs], pos0, rows), 1, tk, tv)
    at = 0
    for (host, kv), p, r in zip(pairs, pos0, rows):
        put_rows(host, 1, p, 0, k[at: at + r])
        put_rows(host, 1, p, 1, v[at: at + r])
        at += r
        same_bytes(host, kv, f"position {p}, {r} rows")
        assert kv.length == 0


def test_special_groups_are_written_as_the_formula_says():
    x = np.zeros((12, 2, 128), np.float32)
    x[0] = -7.5                                  # one number: scale 0
    x[1, 0, 3] = np.inf
    x[1, 1, 100] = -np.inf
    x[2, 0, 64] = np.nan
    x[3, 0, 0], x[3, 0, 1] = 3e38, -3e38         # max - min overflows
    x[4, :, :] = np.float32(2.0) ** -133 * np.arange(128)   # subnormal numbers and scales
    x[5, :, ::2] = -0.0
    x[6, :, 0] = np.float32(2.0) ** -133         # a scale that rounds to 0
    x[7] = np.arange(128) * 0.5 - 16             # quotients on and next to halves
    x[8] = 1e30 * np.arange(128)
    x[9, :, 127] = 1e-20
    x[10, :, 0] = 1.69e38
    x[10, :, 1] = -1.69e38                       # the widest span but one
    x[11] = np.float32(2.0) ** -126 * (1 + np.arange(128))
    x = ref.from_bits(ref.bf16_bits(x))
    host, kv = make(1, 2, 12)
    tfl.tfl_kv4_write(tfl.KV4Rows([kv], [0], [12]), 0, cuda_bf16(x), cuda_bf16(x[::-1].copy()))
    put_rows(host, 0, 0, 0, x)
    put_rows(host, 0, 0, 1, x[::-1])
    for kind in range(2):  # zeros compare equal whatever their sign
        got = ref.Cache(1, 2, 12)
        got.bytes[:] = kv.buffer.cpu().numpy()
        a, s, z = got.get(0, 12, kind)
        b, t, y = host.get(0, 12, kind)
        assert (a == b).all()
        np.testing.assert_array_equal(s, t)
        np.testing.assert_array_equal(z, y)


# ---- read -------------------------------------------------------------------------------

@pytest.mark.parametrize("n_kv,cap,pos0,rows", WRITES)
@pytest.mark.parametrize("strided", [False, True])
def test_rows_read_back_are_what_the_codes_stand_for(n_kv, cap, pos0, rows, strided):
    r = np.random.default_rng(3)
    table = r.permutation((cap + 127) // 128).astype(np.int32)
    pairs = [make(2, n_kv, cap, 0xFF, table) for _ in pos0]
    n = sum(rows)
    want, at = np.full((2, n, n_kv, 128), np.nan), 0
    for (host, kv), p, m in zip(pairs, pos0, rows):
        for kind in range(2):
            x = rows_like_keys(10 + kind + at, m, n_kv)
            put_rows(host, 1, p, kind, x)
            want[kind, at: at + m] = ref.values(*ref.quantise(x))
        at += m
        kv.buffer.copy_(torch.from_numpy(host.bytes))
    wide = torch.full((n + 1, 3, n_kv, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    if strided:
        tk, tv = wide[:, 0], wide[:, 2]
    else:
        tk, tv = wide.new_full((n + 1, n_kv, 128), 7.0), wide.new_full((n + 1, n_kv, 128), 7.0)
    tfl.tfl_kv4_read(tfl.KV4Rows([kv for _, kv in pairs], pos0, rows), 1, tk, tv)
    for got, w in ((tk, want[0]), (tv, want[1])):
        g = host_f32(got)
        assert (g[n:] == 7.0).all()                                     # rows behind the last: left as they were
        # one rounding to bf16 (2^-8 of the value) after one to fp32 (2^-24)
        assert (np.abs(g[:n] - w) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(w) + 1e-38).all()
    if strided:
        assert (host_f32(wide[:, 1]) == 7.0).all()


def test_write_then_read_is_half_a_scale_from_the_rows():
    x, y = rows_like_keys(5, 500, 8), rows_like_keys(6, 500, 8)
    kv = tfl.KV4(1, 8, 1000)
    b = tfl.KV4Rows([kv], [300], [500])
    tfl.tfl_kv4_write(b, 0, cuda_bf16(x), cuda_bf16(y))
    k = torch.empty((500, 8, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    tfl.tfl_kv4_read(b, 0, k, v)
    for got, want in ((k, x), (v, y)):
        _, scale, _ = ref.quantise(want)
        s = np.repeat(scale, 64, -1).astype(np.float64)
        g = host_f32(got)
        # half a scale, the scale's rounding over 15 codes (15 x 2^-8 / 2 doubled), the rounding to bf16
        assert (np.abs(g - want) <= s * (0.5 + 15 * 2.0 ** -8) + 2.0 ** -8 * np.abs(g)).all()


# ---- attention -----------------------------------------------------------------------------

def filled(seed, n_kv, cap, n, layers=1, layer=0, table=None, fill=0xFF):
    """A cache whose positions 0..n-1 hold rows; everything else is `fill` (0xFF: NaN scales and zeros)."""
    host, kv = make(layers, n_kv, cap, fill, table)
    k, v = rows_like_keys(seed, n, n_kv), rows_like_keys(seed + 1, n, n_kv)
    b = tfl.KV4Rows([kv], [0], [n])
    tfl.tfl_kv4_write(b, layer, cuda_bf16(k), cuda_bf16(v))
    return kv, ref.quantise(k), ref.quantise(v)


def queries(seed, n, n_q, std=1.2):
    return ref.from_bits(ref.bf16_bits((std * np.random.default_rng(seed).normal(size=(n, n_q, 128))).astype(np.float32)))


def attend(attn, kvs, pos0, rows, q, layer=0, stream=None):
    n = sum(rows)
    out = torch.full((n + 1, q.shape[1] * 128), 3.0, dtype=torch.bfloat16, device="cuda")
    tfl.tfl_kv4_attention(attn, tfl.KV4Rows(kvs, pos0, rows), layer, cuda_bf16(q).view(-1, q.shape[1] * 128), out, stream)
    got = host_f32(out)
    assert tfl.tfl_kv4_attn_status(attn) == tfl.TFL_OK
    assert (got[n] == 3.0).all()
    return got[:n].reshape(n, q.shape[1], 128)


def check(got, q, pos, kq, vq, what=""):
    for i, p in enumerate(pos):
        out, bound = ref.attention(q[i].astype(np.float64), p, kq, vq)
        err = np.abs(got[i] - out) / bound
        assert np.isfinite(got[i]).all() and err.max() <= 1.0, f"{what} position {p}: {err.max():.2f} bounds"


@pytest.mark.parametrize("n_q,n_kv", [(56, 8), (8, 1), (16, 1), (1, 1), (4, 4), (12, 4), (6, 2), (15, 3)])
@pytest.mark.parametrize("pos", [0, 1, 15, 16, 17, 63, 64, 127, 128, 200, 511, 512, 1000])
def test_one_row_attention_by_heads_and_length(n_q, n_kv, pos):
    kv, kq, vq = filled(20 + pos, n_kv, pos + 1, pos + 1)
    attn = tfl.KV4Attention(n_q, n_kv, max_rows=1, max_positions=pos + 1)
    q = queries(pos, 1, n_q)
    check(attend(attn, [kv], [pos], [1], q), q, [pos], kq, vq)


@pytest.mark.parametrize("n_q,n_kv", [(56, 8), (8, 1), (6, 2), (16, 1)])
@pytest.mark.parametrize("pos0,rows", [(0, 16), (1, 7), (120, 16), (505, 16), (1015, 2), (700, 3), (2040, 9)])
def test_window_attention(n_q, n_kv, pos0, rows):
    kv, kq, vq = filled(30 + pos0, n_kv, pos0 + rows + 40, pos0 + rows, table=None)
    attn = tfl.KV4Attention(n_q, n_kv, max_rows=rows, max_positions=pos0 + rows + 300)
    q = queries(pos0, rows, n_q)
    check(attend(attn, [kv], [pos0], [rows], q), q, range(pos0, pos0 + rows), kq, vq)


def test_long_context_and_permuted_pages():
    n = 20001
    table = np.random.default_rng(8).permutation((n + 127) // 128).astype(np.int32)
    kv, kq, vq = filled(40, 2, n, n, layers=2, layer=1, table=table)
    attn = tfl.KV4Attention(14, 2, max_rows=2, max_positions=n)
    q = queries(9, 2, 14, 0.3)
    check(attend(attn, [kv], [n - 2], [2], q, layer=1), q, [n - 2, n - 1], kq, vq)


def test_sharp_and_flat_softmaxes_and_value_scales_that_differ():
    """Weights from one key to all alike, value groups whose scales span 2^60, and scores that grow along
    the keys (so that the running maximum keeps moving)."""
    n, n_kv = 1300, 1
    k, v = rows_like_keys(50, n, n_kv), rows_like_keys(51, n, n_kv)
    v *= (2.0 ** np.random.default_rng(52).integers(-30, 30, (n, 1, 1))).astype(np.float32)
    k[:, 0, 0] = np.linspace(-40, 90, n)
    k = ref.from_bits(ref.bf16_bits(k))
    _, kv = make(1, n_kv, n)
    tfl.tfl_kv4_write(tfl.KV4Rows([kv], [0], [n]), 0, cuda_bf16(k), cuda_bf16(v))
    q = queries(53, 1, 8)
    q[0, :, 0] = [0, 1, 4, 16, -16, 64, -64, 0]
    q[0, 7] = 0
    attn = tfl.KV4Attention(8, 1, max_rows=1, max_positions=n)
    check(attend(attn, [kv], [n - 1], [1], q), q, [n - 1], ref.quantise(k), ref.quantise(v))


@pytest.mark.parametrize("up,value", [(110, 104), (-110, -80), (0, 104), (60, -110)])
def test_queries_and_values_far_from_one(up, value):
    """Queries times 2^up with keys times 2^-up (the scores stay as they are), values times 2^value."""
    n = 300
    k, v = rows_like_keys(55, n, 2), rows_like_keys(56, n, 2)
    k, v = k * np.float32(2.0 ** -up), v * np.float32(2.0 ** value)  # exact: bf16 numbers
    _, kv = make(1, 2, n)
    tfl.tfl_kv4_write(tfl.KV4Rows([kv], [0], [n]), 0, cuda_bf16(k), cuda_bf16(v))
    q = queries(57, 1, 14) * np.float32(2.0 ** up)
    attn = tfl.KV4Attention(14, 2, max_rows=1, max_positions=n)
    check(attend(attn, [kv], [n - 1], [1], q), q, [n - 1], ref.quantise(k), ref.quantise(v))


def test_streams_of_different_lengths_in_one_call():
    pos0, rows = [0, 15, 1023, 700, 130, 0, 511], [1, 7, 2, 0, 16, 3, 1]
    kvs, qs = [], []
    for s, (p, r) in enumerate(zip(pos0, rows)):
        kvs.append(filled(60 + 2 * s, 8, p + max(r, 1), p + max(r, 1)))
    q = queries(61, sum(rows), 56)
    attn = tfl.KV4Attention(56, 8, max_rows=64, max_positions=1100)
    got = attend(attn, [c[0] for c in kvs], pos0, rows, q)
    at = 0
    for (kv, kq, vq), p, r in zip(kvs, pos0, rows):
        check(got[at: at + r], q[at: at + r], range(p, p + r), kq, vq)
        at += r


def test_rows_do_not_depend_on_what_they_run_with():
    """One-row calls, a window, a batch and larger objects give the same bits."""
    pos0, rows = 1017, 12
    kv, _, _ = filled(70, 8, 2000, pos0 + rows)
    other, _, _ = filled(72, 8, 500, 400)
    q = queries(71, rows + 3, 56)
    small = tfl.KV4Attention(56, 8, max_rows=1, max_positions=pos0 + rows)
    large = tfl.KV4Attention(56, 8, max_rows=64, max_positions=9000)
    single = np.concatenate([attend(small, [kv], [pos0 + i], [1], q[i: i + 1]) for i in range(rows)])
    window = attend(large, [kv], [pos0], [rows], q[:rows])
    batch = attend(large, [other, kv], [300, pos0], [3, rows], np.concatenate([q[rows:], q[:rows]]))[3:]
    shared = attend(large, [kv, kv], [pos0, pos0 + 5], [5, rows - 5], q[:rows])
    assert (single == window).all() and (single == batch).all() and (single == shared).all()


def test_a_key_or_value_that_is_not_a_number_reaches_only_rows_that_attend_it():
    n, at = 300, 290
    for kind in range(2):
        k, v = rows_like_keys(80, n, 2), rows_like_keys(81, n, 2)
        (k, v)[kind][at, 0, 3] = np.nan
        _, kv = make(1, 2, n)
        tfl.tfl_kv4_write(tfl.KV4Rows([kv], [0], [n]), 0, cuda_bf16(k), cuda_bf16(v))
        attn = tfl.KV4Attention(8, 2, max_rows=16, max_positions=n)
        q = queries(82, 10, 8)
        got = attend(attn, [kv], [at - 4], [10], q)
        seen = np.arange(at - 4, at + 6) >= at
        group = slice(0, 64) if kind else slice(0, 128)  # a value's NaN stays in its group's dims
        assert np.isfinite(got[~seen]).all() and np.isfinite(got[:, 4:]).all()
        assert np.isnan(got[seen][:, :4, group]).all()
        if kind:
            assert np.isfinite(got[seen][:, :4, 64:]).all()


def test_strided_queries_and_outputs():
    kv, kq, vq = filled(90, 2, 600, 600)
    q = queries(91, 5, 10)
    wide = torch.full((5, 3, 10 * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 1] = cuda_bf16(q).view(5, -1)
    out = torch.full((7, 2, 10 * 128), 3.0, dtype=torch.bfloat16, device="cuda")
    attn = tfl.KV4Attention(10, 2, max_rows=5, max_positions=600)
    tfl.tfl_kv4_attention(attn, tfl.KV4Rows([kv], [595], [5]), 0, wide[:, 1], out[:, 0])
    got = host_f32(out)
    check(got[:5, 0].reshape(5, 10, 128), q, range(595, 600), kq, vq)
    assert (got[:, 1] == 3.0).all() and (got[5:] == 3.0).all()


def test_captured_calls_replay_on_new_contents():
    n = 700
    kv, _, _ = filled(100, 8, n, n)
    attn = tfl.KV4Attention(56, 8, max_rows=1, max_positions=n)
    k, v = cuda_bf16(rows_like_keys(101, 1, 8)), cuda_bf16(rows_like_keys(102, 1, 8))
    q = cuda_bf16(queries(103, 1, 56)).view(1, -1)
    out, back = torch.zeros_like(q), torch.zeros_like(k)
    row = tfl.KV4Rows([kv], [n - 1], [1])
    st = torch.cuda.Stream()

    def step():
        tfl.tfl_kv4_write(row, 0, k, v)
        tfl.tfl_kv4_attention(attn, row, 0, q, out)
        tfl.tfl_kv4_read(row, 0, back, v_back)

    v_back = torch.zeros_like(v)
    with torch.cuda.stream(st):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step()
    for seed in (110, 120):
        k.copy_(cuda_bf16(rows_like_keys(seed, 1, 8)))
        v.copy_(cuda_bf16(rows_like_keys(seed + 1, 1, 8)))
        q.copy_(cuda_bf16(queries(seed + 2, 1, 56)).view(1, -1))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), back.clone(), v_back.clone()
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (out, back, v_back)):
            assert torch.equal(a, b)


def test_two_objects_on_two_streams_at_once():
    n = 3000
    kv, kq, vq = filled(130, 8, n, n)
    q = [queries(131 + i, 1, 56) for i in range(2)]
    tq = [cuda_bf16(x).view(1, -1) for x in q]
    attn = [tfl.KV4Attention(56, 8, max_rows=1, max_positions=n) for _ in range(2)]
    out = [torch.zeros((1, 56 * 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            tfl.tfl_kv4_attention(attn[i], tfl.KV4Rows([kv], [n - 1], [1]), 0, tq[i], out[i], streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        check(host_f32(out[i]).reshape(1, 56, 128), q[i], [n - 1], kq, vq)


@pytest.mark.parametrize("captured", [False, True])
def test_calls_that_follow_each_other_and_other_streams(captured):
    """Write, read and attention chained through their buffers, with work of torch and of another stream between."""
    n, reps = 1500, 6
    kv, _, _ = filled(135, 8, n + reps, n)
    attn = tfl.KV4Attention(56, 8, max_rows=1, max_positions=n + reps)
    k0, v0 = cuda_bf16(rows_like_keys(136, 1, 8)), cuda_bf16(rows_like_keys(137, 1, 8))
    q0 = cuda_bf16(queries(138, 1, 56)).view(1, -1)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    k, v, q, out = k0.clone(), v0.clone(), q0.clone(), torch.zeros_like(q0)
    big = torch.zeros(1 << 26, device="cuda")

    def chain(slow):
        k.copy_(k0), v.copy_(v0), q.copy_(q0)
        for i in range(reps):
            r = tfl.KV4Rows([kv], [n + i], [1])
            tfl.tfl_kv4_write(r, 0, k, v)
            tfl.tfl_kv4_read(r, 0, k, v)                                   # the next write's rows
            tfl.tfl_kv4_attention(attn, r, 0, q, out)
            if slow:                                                       # the side stream has the next query, late
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    big.add_(1)
                    q.copy_(out)
                torch.cuda.current_stream().wait_stream(side)
            else:
                q.copy_(out)
            tfl.tfl_kv4_attention(attn, r, 0, q, out)
            tfl.tfl_kv4_attention(attn, r, 0, out.clone(), q)

    with torch.cuda.stream(main):
        chain(True)
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=main):
            chain(True)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
    got = out.clone(), q.clone(), kv.buffer.clone()
    assert tfl.tfl_kv4_attn_status(attn) == tfl.TFL_OK
    out.zero_()
    chain(False)                                                           # the legacy stream, in full order
    torch.cuda.synchronize()
    for a, b in zip(got, (out, q, kv.buffer)):
        assert torch.equal(a, b)


# ---- refusals ----------------------------------------------------------------------------

def test_calls_that_are_refused_change_nothing():
    n_kv, cap = 2, 256
    host, kv = make(1, n_kv, cap)
    same = make(1, 3, cap)[1]
    k = torch.zeros((cap + 8, n_kv, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    q = torch.zeros((64, 8 * 128), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    attn = tfl.KV4Attention(8, n_kv, max_rows=8, max_positions=200)

    def refused(code, call, *a):
        with pytest.raises(tfl.TflError) as e:
            call(*a)
        assert e.value.code == code, str(e.value)

    rows = tfl.KV4Rows
    for call in (tfl.tfl_kv4_write, tfl.tfl_kv4_read):
        refused(tfl.TFL_E_CAPACITY, call, rows([kv], [cap], [1]), 0, k, v)
        refused(tfl.TFL_E_CAPACITY, call, rows([kv], [-1], [1]), 0, k, v)
        refused(tfl.TFL_E_CAPACITY, call, rows([kv], [0], [cap + 1]), 0, k, v)
        refused(tfl.TFL_E_ARG, call, rows([kv], [0], [-1]), 0, k, v)
        refused(tfl.TFL_E_ARG, call, rows([kv], [0], [1]), 1, k, v)
        refused(tfl.TFL_E_ARG, call, rows([kv], [0], [1]), -1, k, v)
        refused(tfl.TFL_E_ARG, call, rows([kv, same], [0, 0], [1, 1]), 0, k, v)
        with pytest.raises(ValueError):
            call(rows([kv], [0], [1]), 0, k.float(), v)
        with pytest.raises(ValueError):
            call(rows([kv], [0], [cap]), 0, k[:5], v[:5])
    refused(tfl.TFL_E_ARG, tfl.tfl_kv4_write, rows([kv, kv], [0, 4], [1, 1]), 0, k, v)
    refused(tfl.TFL_E_ARG, tfl.tfl_kv4_read, rows([kv], [0], [1]), 0, k, k)
    big = 1 << 30
    refused(tfl.TFL_E_CAPACITY, tfl.tfl_kv4_write, rows([kv], [2 ** 31 - 1], [1]), 0, k, v)
    with pytest.raises(ValueError):
        tfl.tfl_kv4_write(rows([kv], [0], [big]), 0, k, v)
    at = tfl.tfl_kv4_attention
    refused(tfl.TFL_E_CAPACITY, at, attn, rows([kv], [200], [1]), 0, q, out)      # past the object's positions
    refused(tfl.TFL_E_ARG, at, attn, rows([kv], [0], [9]), 0, q, out)             # past its rows
    refused(tfl.TFL_E_ARG, at, attn, rows([kv], [0], [17]), 0, q, out)
    refused(tfl.TFL_E_ARG, at, attn, rows([same], [0], [1]), 0, q, out)           # other heads
    with pytest.raises(ValueError):
        at(attn, rows([kv], [0], [1]), 0, q[:, :1000], out)
    L, one = tfl.lib(), (ctypes.c_int * 1)(1)
    r = rows([kv], [0], [1])
    for p, ld in ((k.data_ptr() + 2, 256), (k.data_ptr(), 248), (k.data_ptr(), 260)):
        assert L.tfl_kv4_write(r.handles, 1, 0, r.pos0, r.rows, p, v.data_ptr(), ld, None) == tfl.TFL_E_ARG
    assert L.tfl_kv4_attention(attn.handle, r.handles, 1, 0, r.pos0, r.rows, q.data_ptr() + 8, 1024, out.data_ptr(),
                               1024, None) == tfl.TFL_E_ARG
    assert L.tfl_kv4_attention(attn.handle, r.handles, 1, 0, r.pos0, r.rows, q.data_ptr(), 1024, out.data_ptr(),
                               1020, None) == tfl.TFL_E_ARG
    for keep in (-1, cap + 1):
        with pytest.raises(tfl.TflError):
            kv.reset(keep)
    with pytest.raises(ValueError):
        rows([kv], [0, 1], [1])
    torch.cuda.synchronize()
    same_bytes(host, kv)
    # a call without rows is fine and does nothing
    tfl.tfl_kv4_write(rows([kv], [0], [0]), 0, k, v)
    at(attn, rows([kv, kv], [0, 9], [0, 0]), 0, q, out)
    torch.cuda.synchronize()
    same_bytes(host, kv)


def test_queries_and_output_in_one_place_are_refused():
    kv, _, _ = filled(175, 2, 40, 40)
    q = torch.zeros((1, 8 * 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(tfl.TflError) as e:
        tfl.tfl_kv4_attention(tfl.KV4Attention(8, 2, 1, 40), tfl.KV4Rows([kv], [39], [1]), 0, q, q)
    assert e.value.code == tfl.TFL_E_ARG


def test_table_entries_outside_the_cache_are_not_followed():
    """Pages 1 and 3 of five outside: rows there are not written, rows that attend page 0 alone are as ever, reads and longer
    rows end."""
    n_kv, n = 2, 600
    table = np.array([4, 5, 0, -7, 2], np.int32)
    host, kv = make(1, n_kv, n, 0x11, table)
    k, v = rows_like_keys(176, n, n_kv), rows_like_keys(177, n, n_kv)
    tfl.tfl_kv4_write(tfl.KV4Rows([kv], [0], [n]), 0, cuda_bf16(k), cuda_bf16(v))
    for a, b in ((0, 128), (256, 384), (512, 600)):
        put_rows(host, 0, a, 0, k[a:b])
        put_rows(host, 0, a, 1, v[a:b])
    same_bytes(host, kv)
    gk = torch.empty((n, n_kv, 128), dtype=torch.bfloat16, device="cuda")
    gv = torch.empty_like(gk)
    tfl.tfl_kv4_read(tfl.KV4Rows([kv], [0], [n]), 0, gk, gv)
    torch.cuda.synchronize()
    q = queries(178, 1, 8)
    attn = tfl.KV4Attention(8, n_kv, max_rows=2, max_positions=n)
    check(attend(attn, [kv], [127], [1], q), q, [127], ref.quantise(k), ref.quantise(v))
    attend(attn, [kv], [n - 1], [1], q)


# ---- long caches: partials joined in groups -------------------------------------------------

@pytest.mark.parametrize("pos0", [8186, 16378, 511 - 6])
def test_windows_across_a_group_of_units_equal_single_rows_call_after_call(pos0):
    """Rows on both sides of a change of the units' length, number and groups, several calls of one object."""
    rows = 12
    kv, kq, vq = filled(140, 2, pos0 + rows, pos0 + rows)
    q = queries(141, rows, 14)
    attn = tfl.KV4Attention(14, 2, max_rows=16, max_positions=pos0 + 1000)
    window = attend(attn, [kv], [pos0], [rows], q)
    for i in range(rows):
        assert (attend(attn, [kv], [pos0 + i], [1], q[i: i + 1])[0] == window[i]).all()
    assert (attend(attn, [kv], [pos0], [rows], q) == window).all()
    check(window[::11], q[::11], [pos0, pos0 + 11], kq, vq)


def test_the_longest_capacity_and_positions_past_2_gib():
    """Positions whose byte offsets pass 32 bits: 64 heads, the last layer's tile of a 300,000-position cache."""
    n_kv, cap, layers = 64, 300000, 2
    kv = tfl.KV4(layers, n_kv, cap)
    assert kv.buffer.numel() > 2 ** 32
    pos0, n = cap - 20, 20
    k, v = rows_like_keys(150, n, n_kv), rows_like_keys(151, n, n_kv)
    b = tfl.KV4Rows([kv], [pos0], [n])
    tfl.tfl_kv4_write(b, 1, cuda_bf16(k), cuda_bf16(v))
    gk = torch.empty((n, n_kv, 128), dtype=torch.bfloat16, device="cuda")
    gv = torch.empty_like(gk)
    tfl.tfl_kv4_read(b, 1, gk, gv)
    for got, x in ((gk, k), (gv, v)):
        w = ref.values(*ref.quantise(x))
        assert (np.abs(host_f32(got) - w) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(w)).all()
    # the same last keys under every earlier position zero: all earlier keys score 0 and stand for 0
    kv.buffer[((cap + 127) // 128 * 4 + 255) // 256 * 256:].zero_()
    tfl.tfl_kv4_write(b, 1, cuda_bf16(k), cuda_bf16(v))
    attn = tfl.KV4Attention(n_kv, n_kv, max_rows=1, max_positions=cap)
    q = queries(152, 1, n_kv)
    got = attend(attn, [kv], [cap - 1], [1], q, layer=1)
    kq, vq = values64(k), values64(v)
    for h in range(n_kv):
        s = np.concatenate([np.zeros(pos0), kq[:, h] @ q[0, h].astype(np.float64) / np.sqrt(128)])
        p = np.exp(s - s.max())
        p /= p.sum()
        want = p[pos0:] @ vq[:, h]
        # the reference's bound with V zero before pos0: 2^-8 and 2^-7 of sum P |V|'s terms (|z| + s n <= 3 max |x| here)
        tol = 2.0 ** -7 * np.abs(want) + 2.0 ** -10 * (p[pos0:] @ (3 * np.abs(v[:, h]).max() * np.ones((n, 128))))
        assert (np.abs(got[0, h] - want) <= tol).all()


def values64(x):
    return ref.values(*ref.quantise(x))


def test_many_units_on_single_warps_equal_few_units_on_whole_ctas():
    """Calls of few and of many (unit, KV head) pairs, of one tile of columns and of two: the same bits."""
    n_kv, pos0, rows = 64, 8300, 9
    kv, kq, vq = filled(160, n_kv, pos0 + rows, pos0 + rows)
    q = queries(161, rows, n_kv)
    attn = tfl.KV4Attention(n_kv, n_kv, max_rows=16, max_positions=pos0 + rows)
    window = attend(attn, [kv], [pos0], [rows], q)                     # two tiles
    one = attend(attn, [kv], [pos0], [8], q[:8])                       # one tile x 64 heads
    several = attend(attn, [kv] * 9, [pos0 + i for i in range(9)], [1] * 9, q)
    assert (one == window[:8]).all() and (several == window).all()
    check(window[:1], q[:1], [pos0], kq, vq)
    kv8, _, _ = filled(162, 8, 70000, 70000)                           # units of 10 steps, which begin anywhere in a page
    q8 = queries(163, 2, 56)
    few = tfl.KV4Attention(56, 8, max_rows=16, max_positions=70000)
    for p in (69999, 66047, 66048, 65600):
        w = attend(few, [kv8], [p - 1], [2], q8)                       # two tiles
        for i in range(2):
            assert (attend(few, [kv8], [p - 1 + i], [1], q8[i: i + 1])[0] == w[i]).all()


def test_codes_next_to_halves_and_of_every_scale():
    """Numbers whose quotient lies on and next to a half, at scales over the whole range: the codes of the fp32 division."""
    r = np.random.default_rng(170)
    n = 4000
    x = np.zeros((n, 1, 128), np.float32)
    for i in range(n):
        s = ref.from_bits(ref.bf16_bits(np.float32(2.0) ** r.integers(-120, 110) * np.float32(1 + r.integers(0, 128) / 128)))
        with np.errstate(all="ignore"):
            x[i, 0] = s * (r.integers(0, 31, 128).astype(np.float32) / 2 + r.integers(-2, 3, 128).astype(np.float32) * np.float32(2.0) ** -r.integers(4, 9))
            x[i, 0, [0, 64]], x[i, 0, [1, 65]] = 0, 15 * s
    x = ref.from_bits(ref.bf16_bits(x))
    x[::2] -= 2 * np.abs(x[::2]).max(-1, keepdims=True)
    x = ref.from_bits(ref.bf16_bits(x))
    host, kv = make(1, 1, n)
    tfl.tfl_kv4_write(tfl.KV4Rows([kv], [0], [n]), 0, cuda_bf16(x), cuda_bf16(-x))
    got = ref.Cache(1, 1, n)
    got.bytes[:] = kv.buffer.cpu().numpy()
    for kind, y in enumerate((x, -x)):
        a, s, z = got.get(0, n, kind)
        code, scale, zero = ref.quantise(y)
        np.testing.assert_array_equal(s, scale)
        np.testing.assert_array_equal(z, zero)
        np.testing.assert_array_equal(a, code)


@pytest.mark.parametrize("pos0", [3584 - 7, 4480 - 7, 8192 - 3])
def test_windows_across_a_change_of_the_units_length(pos0):
    """64 heads: units of 4, 5, 6 steps before and after 3,584 and 4,480, of 10 around 8,192; a permuted table."""
    n_kv, rows = 64, 16
    table = np.random.default_rng(1).permutation((pos0 + rows + 127) // 128).astype(np.int32)
    kv, kq, vq = filled(180, n_kv, pos0 + rows, pos0 + rows, table=table)
    q = queries(181, rows, n_kv)
    attn = tfl.KV4Attention(n_kv, n_kv, max_rows=32, max_positions=pos0 + rows)
    window = attend(attn, [kv], [pos0], [rows], q)
    for i in (0, 2, 3, 6, 7, 15):
        assert (attend(attn, [kv], [pos0 + i], [1], q[i: i + 1])[0] == window[i]).all()
    twice = attend(attn, [kv, kv], [pos0, pos0], [rows, rows], np.concatenate([q, q]))  # each cut in two
    assert (twice[:rows] == window).all() and (twice[rows:] == window).all()
    check(window[[0, 15]], q[[0, 15]], [pos0, pos0 + 15], kq, vq)


@pytest.mark.parametrize("pos0,rows", [
    ([0, 31, 3583, 8185, 20000], [1, 7, 2, 16, 5]),    # units of two lengths: shared by steps
    ([8190, 7000, 8190, 7001, 8000, 7777, 8190, 8191, 6000, 8190, 7999, 8190, 7400, 8190, 8100, 8190], [1] * 16),
    ([4096, 0, 4090], [16, 1, 1]),                     # one length, shared by units or by steps
    ([20000, 4, 20000], [16, 0, 16]),                  # more units than warps over one cache
])
def test_batches_on_a_full_grid_equal_each_stream_alone(pos0, rows):
    n = max(p + r for p, r in zip(pos0, rows))
    kv, kq, vq = filled(190, 8, n, n)
    q = queries(191, sum(rows), 56)
    attn = tfl.KV4Attention(56, 8, max_rows=64, max_positions=n)
    got = attend(attn, [kv] * len(pos0), pos0, rows, q)
    at = 0
    for p, r in zip(pos0, rows):
        if r:
            assert (attend(attn, [kv], [p], [r], q[at: at + r]) == got[at: at + r]).all()
            check(got[at: at + 1], q[at: at + 1], [p], kq, vq)
        at += r
