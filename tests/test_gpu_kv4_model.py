"""The forward over 4-bit caches on the GPU: a step and a prompt chunk equal, bit for bit, the
same model run operation by operation (each checked on its own elsewhere) with keys and values
quantised, read back and attended through the 4-bit entry points; windows equal one-row steps,
concurrent streams solo ones, resumed prompts fresh ones."""
import pytest
import torch

from gqa_decoder_forward_gb300 import synth, tfl
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu
S = synth.TINY
MAXP = 900


@pytest.fixture(scope="module")
def tiny():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gqa_decoder_forward_gb300 import build
    build.build()
    w = synth.model_weights(S, 41, "cuda")
    m = tfl.Model(S, w, max_rows=256, max_decode_rows=64, max_context=MAXP)
    return w, m, tfl.KV4Runner(m, max_rows=64, max_positions=MAXP)


def bits(t):
    return t.contiguous().view(torch.int16)


def ids_of(seed, n):
    return synth.uniform_ids(seed, n, S.vocab, "cuda")


def by_operations(w, m, ids, kv, pos0, prompt, n_held=None):
    """The layers and the head on rows ids at positions pos0.., through tfl_layer_op, keys and values going through kv (a KV4)."""
    n, qd = ids.numel(), S.n_q * 128
    h = w["embed"][ids.long()].contiguous()
    plain = m.kv(MAXP)                       # where the QKV operation leaves this call's rows
    attn = tfl.KV4Attention(S.n_q, S.n_kv, max_rows=64, max_positions=MAXP)
    for l in range(S.layers):
        q = torch.empty((n, qd), dtype=torch.bfloat16, device="cuda")
        tfl.tfl_layer_op(m, "norm_qkv_rope", l, h, q, plain, pos0, prompt=prompt)
        k, v = plain.read(l, pos0, n)
        tfl.tfl_kv4_write(tfl.KV4Rows([kv], [pos0], [n]), l, k, v)
        ao = torch.empty_like(q)
        if prompt:
            k, v = (torch.empty((pos0 + n, S.n_kv, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
            tfl.tfl_kv4_read(tfl.KV4Rows([kv], [0], [pos0 + n]), l, k, v)
            plain.write(l, 0, k, v)
            tfl.tfl_layer_op(m, "attention", l, q, ao, plain, pos0, prompt=True)
        else:
            tfl.tfl_kv4_attention(attn, tfl.KV4Rows([kv], [pos0], [n]), l, q, ao)
        tfl.tfl_layer_op(m, "o_residual", l, ao, h, prompt=prompt)
        act = torch.empty((n, S.ffn), dtype=torch.bfloat16, device="cuda")
        tfl.tfl_layer_op(m, "norm_gate_up", l, h, act, prompt=prompt)
        tfl.tfl_layer_op(m, "down_residual", l, act, h, prompt=prompt)
    logits = torch.empty((n, S.vocab), dtype=torch.bfloat16, device="cuda")
    tfl.tfl_head(m, h, logits)
    return logits


def prefilled(r, seed, n, cap=MAXP):
    kv = r.kv(cap)
    kv.buffer.fill_(0xFF)                    # what was never written reads as NaN
    kv = tfl.KV4(S.layers, S.n_kv, cap, buffer=kv.buffer)
    ids = ids_of(seed, n)
    for a in range(0, n, 256):
        r.prefill_chunk(kv, ids[a: a + 256].contiguous())
    assert kv.length == n
    return kv


def logits_of(n):
    return torch.full((n, S.vocab), float("nan"), dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("n", [1, 5, 130])
@pytest.mark.parametrize("before", [0, 200])
def test_prompt_chunk_equals_its_operations(tiny, before, n):
    w, m, r = tiny
    kv = prefilled(r, 1, before) if before else r.kv(MAXP)
    twin = tfl.KV4(S.layers, S.n_kv, MAXP, buffer=kv.buffer.clone())
    ids = ids_of(2, n)
    want = by_operations(w, m, ids, twin, before, True)
    got = logits_of(n)
    r.prefill_chunk(kv, ids, got, all_rows=True)
    assert m.status() == tfl.TFL_OK and kv.length == before + n
    assert torch.equal(bits(got), bits(want)) and torch.equal(kv.buffer, twin.buffer)
    one = logits_of(1)
    kv.reset(before)
    r.prefill_chunk(kv, ids, one)            # the last row's logits alone
    assert torch.equal(bits(one), bits(want[-1:]))


@pytest.mark.parametrize("before,n", [(1, 1), (120, 16), (511, 3), (640, 1)])
def test_step_equals_its_operations(tiny, before, n):
    w, m, r = tiny
    kv = prefilled(r, 3, before)
    twin = tfl.KV4(S.layers, S.n_kv, MAXP, buffer=kv.buffer.clone())
    ids = ids_of(4, n)
    want = by_operations(w, m, ids, twin, before, False)
    got = logits_of(n)
    r.decode_step([kv], ids, [n], got)
    assert m.status() == tfl.TFL_OK and kv.length == before + n
    assert torch.isfinite(got.float()).all()
    assert torch.equal(bits(got), bits(want)) and torch.equal(kv.buffer, twin.buffer)


def test_windows_equal_one_row_steps_and_streams_their_solo_runs(tiny):
    _, m, r = tiny
    lens, rows = [250, 1, 127, 500], [16, 3, 1, 7]
    kvs = [prefilled(r, 10 + s, n) for s, n in enumerate(lens)]
    solo = [tfl.KV4(S.layers, S.n_kv, MAXP, buffer=kv.buffer.clone()) for kv in kvs]
    ids = ids_of(20, sum(rows))
    got = logits_of(sum(rows))
    r.decode_step(kvs, ids, rows, got)
    at = 0
    for kv, n, k in zip(solo, lens, rows):
        kv.reset(n)
        for i in range(k):
            one = logits_of(1)
            r.decode_step([kv], ids[at: at + 1].contiguous(), [1], one)
            assert torch.equal(bits(one), bits(got[at: at + 1])), (n, i)
            at += 1
    for a, b in zip(kvs, solo):
        assert a.length == b.length and torch.equal(a.buffer, b.buffer)


def test_prompt_rows_do_not_depend_on_chunks_and_resume_from_a_kept_prefix(tiny):
    _, m, r = tiny
    ids = ids_of(30, 256)
    fresh, cut = r.kv(MAXP), r.kv(MAXP)
    a, b = logits_of(256), logits_of(256)
    r.prefill_chunk(fresh, ids, a, all_rows=True)
    for p, q in ((0, 100), (100, 101), (101, 256)):
        r.prefill_chunk(cut, ids[p:q].contiguous(), b[p:q], all_rows=True)
    assert torch.equal(bits(a), bits(b))
    cut.reset(77)
    r.prefill_chunk(cut, ids[77:].contiguous(), b[77:], all_rows=True)
    assert torch.equal(bits(a), bits(b))


def test_refusals_leave_the_lengths(tiny):
    _, m, r = tiny
    kv, small = prefilled(r, 50, 60, cap=64), tfl.KV4(S.layers, S.n_kv, 8)
    other = tfl.KV4(S.layers, S.n_kv + 1, 64)
    out, ids = logits_of(64), ids_of(51, 64)

    def refused(code, call, *a, **k):
        with pytest.raises(tfl.TflError) as e:
            call(*a, **k)
        assert e.value.code == code, str(e.value)

    refused(tfl.TFL_E_CAPACITY, r.decode_step, [kv], ids, [5], out)
    refused(tfl.TFL_E_CAPACITY, r.prefill_chunk, kv, ids[:5].contiguous())
    refused(tfl.TFL_E_CAPACITY, r.prefill_chunk, small, ids[:9].contiguous())
    refused(tfl.TFL_E_ARG, r.decode_step, [kv, kv], ids, [1, 1], out)
    refused(tfl.TFL_E_ARG, r.decode_step, [other], ids, [1], out)
    refused(tfl.TFL_E_ARG, r.prefill_chunk, other, ids[:1].contiguous())
    refused(tfl.TFL_E_ARG, r.decode_step, [kv], ids, [0], out)
    refused(tfl.TFL_E_ARG, r.decode_step, [kv], ids, [17], out)
    short = tfl.KV4Runner(m, max_rows=2, max_positions=32)
    refused(tfl.TFL_E_ARG, short.decode_step, [r.kv(64)], ids, [3], out)
    refused(tfl.TFL_E_CAPACITY, short.decode_step, [kv], ids, [1], out)
    refused(tfl.TFL_E_WORKSPACE, short.prefill_chunk, prefilled(r, 52, 200), ids)
    L = tfl.lib()
    h = tfl._kv_array([kv])
    one = (tfl.ctypes.c_int * 1)(1)
    ws = r.step_ws
    for p, n, code in ((0, ws.numel(), tfl.TFL_E_ARG), (ws.data_ptr() + 16, ws.numel(), tfl.TFL_E_ARG),
                       (ws.data_ptr(), ws.numel() - 1, tfl.TFL_E_WORKSPACE)):
        assert L.tfl_decode_step_kv4(m.handle, r.attention.handle, h, 1, ids.data_ptr(), one, out.data_ptr(), p, n, None) == code
    assert L.tfl_decode_step_kv4(m.handle, None, h, 1, ids.data_ptr(), one, out.data_ptr(), ws.data_ptr(), ws.numel(), None) == tfl.TFL_E_ARG
    wrong = tfl.KV4Attention(S.n_q * 2, S.n_kv, max_rows=4, max_positions=64)
    assert L.tfl_decode_step_kv4(m.handle, wrong.handle, h, 1, ids.data_ptr(), one, out.data_ptr(), ws.data_ptr(), ws.numel(), None) == tfl.TFL_E_ARG
    assert kv.length == 60 and small.length == 0
    assert tfl.lib().tfl_kv4_prompt_workspace_bytes(m.handle, MAXP + 1) == 0
    assert tfl.lib().tfl_kv4_step_workspace_bytes(None) == 0


def test_a_33b_layer_steps_over_4_bits():
    """One 33B-shaped layer: a 7-row window equals one-row steps, and the kernels it runs are the 4-bit ones."""
    shape = synth.NANBEIGE_33B.with_layers(1)
    w = gu.layer_weights(shape, 61)
    w["embed"] = synth.layer_weight(synth.NANBEIGE_33B.with_layers(1), 61, 0, "wq", "cuda")[:4096].contiguous()
    # an embedding of 4,096 rows stands in for the vocabulary: ids stay below it, and the head is not read
    w["lm_head"] = torch.zeros(shape.vocab, shape.hidden, dtype=torch.bfloat16, device="cuda")
    w["final_norm"] = torch.ones(shape.hidden, dtype=torch.bfloat16, device="cuda")
    m = tfl.Model(shape, w, max_rows=256, max_decode_rows=16, max_context=1024)
    r = tfl.KV4Runner(m, max_rows=16, max_positions=1024)
    kv, twin = r.kv(1024), r.kv(1024)
    ids = (synth.uniform_ids(62, 207, 4096, "cuda")).to(torch.int32)
    out = torch.empty((7, shape.vocab), dtype=torch.bfloat16, device="cuda")
    for c in (kv, twin):
        r.prefill_chunk(c, ids[:200].contiguous())
    tfl.tfl_profile(m, True)
    r.decode_step([kv], ids[200:].contiguous(), [7], out)
    launched = tfl.tfl_profile_read(m)
    tfl.tfl_profile(m, False)
    assert launched["kv4_write"][1] == 1 and launched["kv4_attention"][1] == 1
    assert launched["attn_decode_block"][1] == 0 and launched["decode_step_persistent"][1] == 0
    for i in range(7):
        r.decode_step([twin], ids[200 + i: 201 + i].contiguous(), [1], out[:1])
    assert m.status() == tfl.TFL_OK
    k, v = (torch.empty((2, 207, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for i, c in enumerate((kv, twin)):
        tfl.tfl_kv4_read(tfl.KV4Rows([c], [0], [207]), 0, k[i], v[i])
    assert torch.equal(bits(k[0]), bits(k[1])) and torch.equal(bits(v[0]), bits(v[1]))
    assert torch.isfinite(k.float()).all()
