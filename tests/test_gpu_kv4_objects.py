"""Objects of the 4-bit cache made while a stream still works on the memory that they take."""
import numpy as np
import pytest
import torch

from gqa_decoder_forward_gb300 import synth, tfl
from tests import kv4_ref as ref
from tests.test_gpu_kv4 import _built, cuda_bf16, put_rows, queries, rows_like_keys  # noqa: F401

pytestmark = pytest.mark.gpu


def busy(stream):
    """Some tens of milliseconds of ordinary work on a stream, so that what follows it there is late."""
    x = torch.ones(1 << 28, device="cuda")
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(40):
            x.add_(1)
    return x


def test_a_cache_over_a_buffer_that_a_side_stream_fills_keeps_its_table():
    n_kv, cap, n = 2, 500, 300
    host = ref.Cache(1, n_kv, cap, 0x5A)
    x, y = rows_like_keys(300, n, n_kv), rows_like_keys(301, n, n_kv)
    k, v = cuda_bf16(x), cuda_bf16(y)
    buf = torch.empty(host.bytes.size, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    held = busy(side)
    with torch.cuda.stream(side):
        buf.fill_(0x5A)
        kv = tfl.KV4(1, n_kv, cap, buffer=buf)
        tfl.tfl_kv4_write(tfl.KV4Rows([kv], [0], [n]), 0, k, v)
    torch.cuda.synchronize()
    del held
    put_rows(host, 0, 0, 0, x)
    put_rows(host, 0, 0, 1, y)
    got = buf.cpu().numpy()
    assert (got[: host.pages * 4].view(np.int32) == np.arange(host.pages)).all()
    assert (got[host.table_bytes:] == host.bytes[host.table_bytes:]).all()


def test_objects_in_memory_that_a_side_stream_still_writes():
    """The caching allocator hands a freed block back to its stream while work on it is pending (the sizes asked for
    again, so as a rule the same blocks)."""
    kv = tfl.KV4(1, 2, 128)
    tfl.tfl_kv4_write(tfl.KV4Rows([kv], [0], [100]), 0, cuda_bf16(rows_like_keys(302, 100, 2)), cuda_bf16(rows_like_keys(303, 100, 2)))
    q = cuda_bf16(queries(304, 1, 8)).view(1, -1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    nbytes = int(tfl.lib().tfl_kv4_attn_bytes(8, 2, 128, 16, 65536))
    table = int(tfl.tfl_kv4_bytes(4, 8, 65536))
    with torch.cuda.stream(side):
        blocks = [torch.empty(nbytes, dtype=torch.uint8, device="cuda"), torch.empty(table, dtype=torch.uint8, device="cuda")]
    held = busy(side)
    with torch.cuda.stream(side):
        for b in blocks:
            b.fill_(0xFF)
        del b, blocks
        attn = tfl.KV4Attention(8, 2, max_rows=16, max_positions=65536)
        big = tfl.KV4(4, 8, 65536)
        out = torch.zeros_like(q)
        tfl.tfl_kv4_attention(attn, tfl.KV4Rows([kv], [99], [1]), 0, q, out)
    torch.cuda.synchronize()
    del held
    assert tfl.tfl_kv4_attn_status(attn, side) == tfl.TFL_OK
    assert (big.buffer[: 512 * 4].cpu().numpy().view(np.int32) == np.arange(512)).all()
    assert torch.isfinite(out.float()).all()
    # the bf16 cache's table in the same way
    w = synth.model_weights(synth.TINY, 5, "cuda")
    m = tfl.Model(synth.TINY, w, max_rows=64, max_decode_rows=4, max_context=4096)
    size = int(tfl.tfl_kv_bytes(m.cfg, 4096))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        block = torch.empty(size, dtype=torch.uint8, device="cuda")
    held = busy(side)
    with torch.cuda.stream(side):
        block.fill_(0xFF)
        del block
        plain = m.kv(4096)
    torch.cuda.synchronize()
    assert (plain.buffer[: 32 * 4].cpu().numpy().view(np.int32) == np.arange(32)).all()


def test_calls_without_rows_take_empty_tensors():
    kv = tfl.KV4(1, 2, 128)
    before = kv.buffer.clone()
    attn = tfl.KV4Attention(8, 2, max_rows=1, max_positions=128)
    none = tfl.KV4Rows([kv, kv], [3, 9], [0, 0])
    k, v = (torch.empty((0, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tfl.tfl_kv4_write(tfl.KV4Rows([kv], [3], [0]), 0, k, v)
    tfl.tfl_kv4_read(none, 0, k, v)
    q = torch.empty((0, 8 * 128), dtype=torch.bfloat16, device="cuda")
    tfl.tfl_kv4_attention(attn, none, 0, q, torch.empty_like(q))
    torch.cuda.synchronize()
    assert torch.equal(kv.buffer, before)


def test_one_row_of_tensors_with_different_strides():
    kv, twin = tfl.KV4(1, 2, 128), tfl.KV4(1, 2, 128)
    kv.buffer[256:].zero_(), twin.buffer[256:].zero_()
    k, v = (cuda_bf16(rows_like_keys(s, 1, 2)) for s in (310, 311))
    wide = torch.zeros((4, 3, 2, 128), dtype=torch.bfloat16, device="cuda")
    wide[:1, 1] = v
    tfl.tfl_kv4_write(tfl.KV4Rows([kv], [7], [1]), 0, k, wide[:, 1])
    tfl.tfl_kv4_write(tfl.KV4Rows([twin], [7], [1]), 0, k, v)
    assert torch.equal(kv.buffer, twin.buffer)


def test_a_runner_for_longer_caches_than_the_models_context():
    w = synth.model_weights(synth.TINY, 6, "cuda")
    m = tfl.Model(synth.TINY, w, max_rows=64, max_decode_rows=4, max_context=200)
    ids = synth.uniform_ids(7, 61, synth.TINY.vocab, "cuda")
    out = [torch.empty((1, synth.TINY.vocab), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for lg, r in zip(out, (tfl.KV4Runner(m, max_rows=4), tfl.KV4Runner(m, max_rows=4, max_positions=200))):
        kv = r.kv(1000)
        r.prefill_chunk(kv, ids[:60].contiguous())
        r.decode_step([kv], ids[60:].contiguous(), [1], lg)
        kv.reset(150)
        with pytest.raises(tfl.TflError) as e:                       # past the model's context
            r.prefill_chunk(kv, ids[:60].contiguous())
        assert e.value.code == tfl.TFL_E_CAPACITY
    assert m.status() == tfl.TFL_OK and torch.equal(out[0].view(torch.int16), out[1].view(torch.int16))


def test_what_workspaces_hold_before_a_call_means_nothing():
    w = synth.model_weights(synth.TINY, 8, "cuda")
    m = tfl.Model(synth.TINY, w, max_rows=64, max_decode_rows=16, max_context=300)
    ids = synth.uniform_ids(9, 150, synth.TINY.vocab, "cuda")
    got = []
    for fill in (0x00, 0xFF):                                        # zeros, and NaN in every type
        r = tfl.KV4Runner(m, max_rows=16, max_positions=300)
        kv = tfl.KV4(synth.TINY.layers, synth.TINY.n_kv, 300, buffer=torch.full_like(r.kv(300).buffer, fill))
        lg = torch.empty((71, synth.TINY.vocab), dtype=torch.bfloat16, device="cuda")
        for a, b in ((0, 64), (64, 127)):
            r.prompt_ws.fill_(fill), r.step_ws.fill_(fill), r.attention.workspace[256:].fill_(fill)
            r.prefill_chunk(kv, ids[a:b].contiguous(), lg[:64], all_rows=True)
        r.prompt_ws.fill_(fill), r.step_ws.fill_(fill), r.attention.workspace[256:].fill_(fill)
        r.decode_step([kv], ids[127:134].contiguous(), [7], lg[64:])
        torch.cuda.synchronize()
        got.append(lg.view(torch.int16).clone())
    assert m.status() == tfl.TFL_OK and torch.equal(got[0], got[1])


@pytest.mark.parametrize("rows", [[1], [3, 1, 7]])
def test_the_forward_on_a_side_stream_and_replayed_equals_the_legacy_streams(rows):
    """On streams of their own the kernels are set up while the ones before still run."""
    w = synth.model_weights(synth.TINY, 10, "cuda")
    m = tfl.Model(synth.TINY, w, max_rows=256, max_decode_rows=16, max_context=600)
    r = tfl.KV4Runner(m, max_rows=16, max_positions=600)
    lens = [250, 40, 500][: len(rows)]
    ids = synth.uniform_ids(11, sum(lens) + sum(rows), synth.TINY.vocab, "cuda")
    side = torch.cuda.Stream()

    def run(kvs, logits, step):
        at = 0
        for kv, n in zip(kvs, lens):
            for a in range(0, n, 256):
                r.prefill_chunk(kv, ids[at + a: at + min(n, a + 256)], logits[:1])
            at += n
        for _ in range(4):                                           # the same rows again: steps that follow each other
            for kv, n in zip(kvs, lens):
                kv.reset(n)
            step(kvs, ids[at:].contiguous(), logits)

    outs, bufs = [], []
    for how in ("legacy", "side", "graph"):
        kvs = [r.kv(600) for _ in rows]
        for kv in kvs:
            kv.buffer[256:].zero_()                                  # five pages: the table is the first 256 bytes
        lg = torch.zeros((sum(rows), synth.TINY.vocab), dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        if how == "legacy":
            run(kvs, lg, lambda k, i, o: r.decode_step(k, i, rows, o))
        elif how == "side":
            with torch.cuda.stream(side):
                run(kvs, lg, lambda k, i, o: r.decode_step(k, i, rows, o))
        else:
            with torch.cuda.stream(side):
                run(kvs, lg, lambda k, i, o: None)
            torch.cuda.synchronize()
            last = ids[sum(lens):].contiguous()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                for _ in range(3):
                    for kv, n in zip(kvs, lens):
                        kv.reset(n)
                    r.decode_step(kvs, last, rows, lg)
            lg.zero_()
            for _ in range(3):
                graph.replay()
        torch.cuda.synchronize()
        assert m.status() == tfl.TFL_OK
        outs.append(lg.view(torch.int16).clone())
        bufs.append([kv.buffer.clone() for kv in kvs])
    for o, b in zip(outs[1:], bufs[1:]):
        assert torch.equal(o, outs[0])
        assert all(torch.equal(x[256:], y[256:]) for x, y in zip(b, bufs[0]))   # behind the table and its padding, which nothing writes
