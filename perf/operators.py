"""The 4-bit key/value cache's operators, case by case: quantising rows as they are
written, reading rows back, and attention over the cache.

`own` False computes them in plain torch; `own` True calls the library
(gqa_decoder_forward_gb300.tfl).  Both work on the same cache bytes, laid out as
include/tfl.h says: a page table (int32 per page, padded to 256 bytes), then for
each (layer, page of 128 positions, head) eight blocks of 16 positions, each block
being 16 rows of key codes, 16 key (scale, zero) pairs, and the same for values.
"""
import math

import torch

own = False

D = 128          # dims of a head
GROUP = 64       # dims that share a scale and a zero
PAGE = 128       # positions of a page
BLOCK = 16       # positions of a block
ROW_W = 8        # a row's codes, in 8-byte words (64 bytes)
BLOCK_W = 288    # a block, in 8-byte words (2,304 bytes): 128 + 16 + 128 + 16
V_W = 144        # where a block's values begin, in 8-byte words


# ---- cases ------------------------------------------------------------------------

def _case(name, op, n_kv, group, pos, rows, fused=False):
    return {"name": name, "op": op, "n_kv": n_kv, "group": group, "pos": ",".join(map(str, pos)),
            "rows": ",".join(map(str, rows)), "fused": fused}


def listed():
    ragged = [8191 - 397 * s for s in range(16)]
    return [
        # one stream's next token, written into one layer of the 33B-shaped cache
        _case("write_1_token", "write", 8, 7, [4099], [1]),
        # sixteen streams' next tokens at their own lengths, keys and values still in the fused projection's rows
        _case("write_16_streams", "write", 8, 7, ragged, [1] * 16, True),
        # a prompt chunk of the largest size, after an 8K prefix
        _case("write_chunk_2048", "write", 8, 7, [8192], [2048], True),
        # a short odd prompt that starts and ends inside a page, tiny model
        _case("read_333_tiny", "read", 1, 8, [77], [333]),
        # an 8K prefix read back before a prompt goes on
        _case("read_8192", "read", 8, 7, [0], [8192]),
        # the longest prefix read back, one layer
        _case("read_131072", "read", 8, 7, [0], [131072]),
        # the tiny model's first tokens after its 64-token prompt: launch latency alone
        _case("attend_tiny_65", "attend", 1, 8, [64], [1]),
        # the next token after 4K
        _case("attend_4096", "attend", 8, 7, [4096], [1]),
        # sixteen streams of about 8K, one row each
        _case("attend_16_streams", "attend", 8, 7, ragged, [1] * 16),
        # the next token after the longest prompt
        _case("attend_131072", "attend", 8, 7, [131071], [1]),
        # a window of guesses over 4K keys, queries still in the fused projection's rows
        _case("attend_window_16", "attend", 8, 7, [4096], [16], True),
        # streams of very different lengths with windows of 1 to 7 rows
        _case("attend_ragged", "attend", 8, 7, [0, 15, 1023, 5000, 12345, 31999], [1, 7, 2, 5, 1, 3]),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend"])
    n_kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    if n_kv * group > 64:
        group = 64 // n_kv
    fused = rng.random() < 0.5
    streams = rng.choice([1, 1, 2, 3, 5, 8, 13, 16])
    if op == "attend":
        left, row_keys, pos, rows = 131072, 131072, [], []
        for s in range(streams):
            ctx = _log(rng, 1, max(1, min(131071, left // (streams - s))))
            r = rng.choice([1, 1, 1, 2, 3, 7, 16])
            while r > 1 and (ctx * r > row_keys // (streams - s) or sum(rows) + r + (streams - s - 1) > 64):
                r -= 1
            pos.append(ctx - 1)
            rows.append(r)
            left -= ctx
            row_keys -= ctx * r
        return {k: v for k, v in _case("", op, n_kv, group, pos, rows, fused).items() if k != "name"}
    most = 2048 if op == "write" else 131072
    if streams == 1:
        pos, rows = [_log(rng, 1, 16384) - 1], [_log(rng, 1, most)]
    else:
        pos = [_log(rng, 1, 16384) - 1 for _ in range(streams)]
        rows = [_log(rng, 1, most // streams) for _ in range(streams)]
    return {k: v for k, v in _case("", op, n_kv, group, pos, rows, fused).items() if k != "name"}


def _ints(text):
    return [int(x) for x in text.split(",")]


def work(case):
    pos, rows, n_kv = _ints(case["pos"]), _ints(case["rows"]), case["n_kv"]
    n, held = sum(rows), 2 * (D // 2 + 2 * 2 * (D // GROUP))  # bytes of one position's key and value in the cache, one head
    dense = 2 * D * 2                                         # the same in bf16
    if case["op"] == "write":   # rows in, codes out; and the values they stand for
        return {"bytes": n * n_kv * (dense + held + dense), "flops": 0}
    if case["op"] == "read":
        return {"bytes": n * n_kv * (held + dense), "flops": 0}
    n_q = n_kv * case["group"]
    keys = sum(p + r for p, r in zip(pos, rows))
    seen = sum(r * p + r * (r + 1) // 2 for p, r in zip(pos, rows))
    return {"bytes": keys * n_kv * held + 2 * n * n_q * D * 2, "flops": 4 * seen * n_q * D}


# ---- the plain form ------------------------------------------------------------------

def _quantise(x):
    """x [..., 128] bf16 -> codes uint8 [..., 128], (scale, zero) float32 [..., 2] each,
    scale and zero being bf16 numbers."""
    g = x.float().unflatten(-1, (D // GROUP, GROUP))
    zero = g.amin(-1)
    span = g.amax(-1) - zero
    bad = ~torch.isfinite(span)
    scale = (span / 15).to(torch.bfloat16).float()
    code = torch.round((g - zero[..., None]) / torch.where(scale > 0, scale, 1.0)[..., None])
    code = torch.where(((scale > 0) & ~bad)[..., None], code, 0.0).clamp(0, 15).to(torch.uint8).flatten(-2)
    return code, torch.where(bad, 0.0, scale), torch.where(bad, float("nan"), zero)


def _halves_swapped(pos, t):
    """t [N, heads, 2, ...]: the two 32-byte halves of a row change places where bit 1 of the position is set."""
    return torch.where(((pos >> 1) & 1).bool().view(-1, 1, *[1] * (t.dim() - 2)), t.flip(2), t)


def _pack(code, pos):
    """codes [N, heads, 128] -> [N, heads, 8] words of 8 bytes: word c holds dims 8c..8c+7, then 64+8c..64+8c+7,
    two codes to a byte, the lower dim in the low half."""
    b = code[..., 0::2] | (code[..., 1::2] << 4)                       # byte i: dims 2i, 2i + 1
    b = b.unflatten(-1, (2, 2, 4, 4)).permute(0, 1, 3, 4, 2, 5)        # [half][word][group][byte]
    return _halves_swapped(pos, b).reshape(*b.shape[:2], 64).contiguous().view(torch.int64)


def _unpack(words, pos):
    """The reverse: [N, heads, 8] words -> codes float32 [N, heads, 128]."""
    b = words.contiguous().view(torch.uint8).unflatten(-1, (2, 4, 2, 4))
    b = _halves_swapped(pos, b).permute(0, 1, 4, 2, 3, 5).reshape(*words.shape[:2], 64)
    return torch.stack((b & 15, b >> 4), -1).flatten(-2).float()


def _places(st, sidx, pos):
    """The first 8-byte word of the blocks that hold (stream, position) for each head, and the row in the block."""
    head = torch.arange(st["n_kv"], device=pos.device)
    tile = (pos // PAGE)[:, None] * st["n_kv"] + head
    base = sidx[:, None] * st["stream_w"] + st["table_w"] + (tile * (PAGE // BLOCK) + (pos % PAGE // BLOCK)[:, None]) * BLOCK_W
    return base, (pos % BLOCK)[:, None]


def _store(st, sidx, pos, k, v):
    mem = st["cache"].view(torch.int64).view(-1)
    base, i = _places(st, sidx, pos)
    w = torch.arange(ROW_W, device=pos.device)
    for at, x in ((base, k), (base + V_W, v)):
        code, scale, zero = _quantise(x)
        mem[(at + i * ROW_W)[..., None] + w] = _pack(code, pos)
        mem[at + BLOCK * ROW_W + i] = torch.stack((scale, zero), -1).to(torch.bfloat16).flatten(-2).contiguous().view(torch.int64)[..., 0]


def _load(st, sidx, pos):
    """Keys and values that the cache stands for, [N, heads, 128] float32."""
    mem = st["cache"].view(torch.int64).view(-1)
    base, i = _places(st, sidx, pos)
    w = torch.arange(ROW_W, device=pos.device)
    got = []
    for at in (base, base + V_W):
        code = _unpack(mem[(at + i * ROW_W)[..., None] + w], pos).unflatten(-1, (D // GROUP, GROUP))
        meta = mem[at + BLOCK * ROW_W + i][..., None].view(torch.bfloat16).float().unflatten(-1, (D // GROUP, 2))
        got.append((code * meta[..., 0, None] + meta[..., 1, None]).flatten(-2))
    return got


def _attend(st):
    """Every stream's rows at once, padded to the longest: softmax(q k / sqrt(128)) v over keys 0..position."""
    S, T, n_kv, G = st["streams"], st["keys"], st["n_kv"], st["group"]
    t = torch.arange(T, device="cuda")
    last = st["pos0"] + st["rows"] - 1                                   # [S]
    sidx = torch.arange(S, device="cuda")[:, None].expand(S, T).reshape(-1)
    held = torch.minimum(t[None, :], last[:, None])                      # past a stream's end: its last key, masked below
    k, v = (x.view(S, T, n_kv, D).permute(0, 2, 1, 3) for x in _load(st, sidx, held.reshape(-1)))
    q = st["q"].float()[st["pad"]].view(S, -1, n_kv, G, D).permute(0, 2, 1, 3, 4).flatten(2, 3)   # [S, n_kv, R * G, D]
    score = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    see = t <= st["pad_pos"][..., None]                                  # [S, R, T]
    score = score.masked_fill(~see.repeat_interleave(G, 1)[:, None], float("-inf"))
    p = torch.exp(score - score.amax(-1, keepdim=True))
    o = (p / p.sum(-1, keepdim=True)) @ v
    o = o.unflatten(2, (-1, G)).permute(0, 2, 1, 3, 4).reshape(-1, n_kv * G * D)
    return o[st["pick"]].to(torch.bfloat16)


# ---- what the tools call ---------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    pos0, rows = _ints(case["pos"]), _ints(case["rows"])
    n_kv, G, S, N = case["n_kv"], case["group"], len(pos0), sum(rows)
    keys = max(p + r for p, r in zip(pos0, rows))
    pages = (keys + PAGE - 1) // PAGE
    table_w = (pages * 4 + 255) // 256 * 32
    stream_w = table_w + pages * n_kv * (PAGE // BLOCK) * BLOCK_W
    cache = torch.full((S, stream_w * 8), 255, dtype=torch.uint8, device="cuda")   # what was never written reads as NaN
    cache[:, : pages * 4] = torch.arange(pages, dtype=torch.int32, device="cuda").view(torch.uint8)
    st = {"op": case["op"], "n_kv": n_kv, "group": G, "streams": S, "keys": keys, "stream_w": stream_w, "table_w": table_w,
          "cache": cache}
    p0, r = torch.tensor(pos0, device="cuda"), torch.tensor(rows, device="cuda")
    st["pos0"], st["rows"] = p0, r
    first = torch.cumsum(r, 0) - r
    st["sidx"] = torch.repeat_interleave(torch.arange(S, device="cuda"), r)
    st["pos"] = torch.arange(N, device="cuda") - first[st["sidx"]] + p0[st["sidx"]]
    # keys: some channels larger than others, as after the rotation; values without such channels
    k_ch, v_ch = 1.7 * torch.exp(0.5 * normal(n_kv, D)), 1.7
    lead = 0 if case["op"] == "write" else 1
    if lead:  # the cache before the call: all positions up to each stream's last, in pieces that bound the index tensors
        for s in range(S):
            for a in range(0, pos0[s] + rows[s], 16384):
                b = min(a + 16384, pos0[s] + rows[s])
                at = torch.arange(a, b, device="cuda")
                _store(st, torch.full_like(at, s), at, (normal(b - a, n_kv, D) * k_ch).to(torch.bfloat16),
                       (normal(b - a, n_kv, D) * v_ch).to(torch.bfloat16))
    width = (G + 2) * n_kv * D
    qkv = torch.empty(N, width, dtype=torch.bfloat16, device="cuda") if case["fused"] else None

    def rows_of(x, a):
        x = x.to(torch.bfloat16)
        if qkv is None:
            return x
        part = qkv[:, a: a + x[0].numel()].unflatten(-1, x.shape[1:])
        part.copy_(x)
        return part

    if case["op"] == "write":
        st["k"] = rows_of(normal(N, n_kv, D) * k_ch, G * n_kv * D)
        st["v"] = rows_of(normal(N, n_kv, D) * v_ch, (G + 1) * n_kv * D)
    if case["op"] == "attend":
        st["q"] = rows_of(1.2 * normal(N, n_kv * G * D), 0)
        R = max(rows)
        i = torch.arange(R, device="cuda")
        inside = torch.minimum(i[None, :], (r - 1)[:, None])             # [S, R]
        st["pad"] = (first[:, None] + inside).reshape(-1)
        st["pad_pos"] = p0[:, None] + inside
        st["pick"] = (st["sidx"] * R + st["pos"] - p0[st["sidx"]])
    if own:
        from gqa_decoder_forward_gb300 import tfl
        st["tfl"] = tfl
        st["kvs"] = [tfl.KV4(1, n_kv, pages * PAGE, buffer=cache[s]) for s in range(S)]
        st["batch"] = tfl.KV4Rows(st["kvs"], pos0, rows)
        st["k_out"] = torch.empty(N, n_kv, D, dtype=torch.bfloat16, device="cuda")
        st["v_out"] = torch.empty_like(st["k_out"])
        if case["op"] == "attend":
            st["attention"] = tfl.KV4Attention(n_kv * G, n_kv, max_rows=N, max_positions=pages * PAGE)
            st["out"] = torch.empty(N, n_kv * G * D, dtype=torch.bfloat16, device="cuda")
    return st


def run(st):
    if own:
        tfl = st["tfl"]
        if st["op"] == "attend":
            tfl.tfl_kv4_attention(st["attention"], st["batch"], 0, st["q"], st["out"])
            return st["out"]
        if st["op"] == "write":
            tfl.tfl_kv4_write(st["batch"], 0, st["k"], st["v"])
        tfl.tfl_kv4_read(st["batch"], 0, st["k_out"], st["v_out"])
        return {"k": st["k_out"], "v": st["v_out"]}
    if st["op"] == "attend":
        return _attend(st)
    if st["op"] == "write":
        _store(st, st["sidx"], st["pos"], st["k"], st["v"])
    k, v = _load(st, st["sidx"], st["pos"])
    return {"k": k.to(torch.bfloat16), "v": v.to(torch.bfloat16)}


# ---- the same in 64 bits, apart from the above ---------------------------------------------

def _exact_rows(x):
    """What a written row stands for: 16 even steps from its group's least to (nearly) its largest value, the step a bf16 number."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for g in range(D // GROUP):
        part = x[..., g * GROUP: (g + 1) * GROUP].double()
        low, high = part.min(-1, keepdim=True).values, part.max(-1, keepdim=True).values
        step = ((high - low) / 15).to(torch.bfloat16).double()
        code = torch.where(step > 0, torch.round((part - low) / step.clamp_min(1e-300)), 0.0).clamp(0, 15)
        out[..., g * GROUP: (g + 1) * GROUP] = low + step * code
    return out


def _exact_held(st, s, head, n, kind):
    """Keys (kind 0) or values (1) of positions 0..n-1 of one stream and head, from the cache's bytes, [n, 128] float64."""
    page = torch.arange((n + PAGE - 1) // PAGE, device="cuda")
    at = st["table_w"] * 8 + (page * st["n_kv"] + head) * PAGE // BLOCK * BLOCK_W * 8
    tile = st["cache"][s][(at[:, None] + torch.arange(PAGE // BLOCK * BLOCK_W * 8, device="cuda")).view(-1)].view(-1, BLOCK_W * 8)
    codes = tile[:, kind * V_W * 8:][:, : BLOCK * 64].reshape(-1, 64)[:n]                    # position by position
    meta = tile[:, kind * V_W * 8 + BLOCK * 64:][:, : BLOCK * 8].reshape(-1, 8)[:n].contiguous().view(torch.bfloat16).double()
    p, d = torch.arange(n, device="cuda")[:, None], torch.arange(D, device="cuda")[None, :]
    chunk, word, code = d % 64 // 8, d // 64, d % 8
    byte = 8 * (chunk ^ (4 * ((p >> 1) & 1))) + 4 * word + code // 2
    value = ((codes.gather(1, byte).to(torch.int64) >> (4 * (code % 2))) & 15).double()
    return meta[:, [1]].where(d < 64, meta[:, [3]]) + meta[:, [0]].where(d < 64, meta[:, [2]]) * value


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    pos0, rows, n_kv, G = _ints(case["pos"]), _ints(case["rows"]), case["n_kv"], case["group"]
    if case["op"] == "write":
        return {"k": _exact_rows(st["k"]), "v": _exact_rows(st["v"])}
    starts = [sum(rows[:s]) for s in range(len(rows))]
    if case["op"] == "read":
        out = [torch.empty(sum(rows), n_kv, D, dtype=torch.float64, device="cuda") for _ in range(2)]
        for s, (p, r) in enumerate(zip(pos0, rows)):
            for h in range(n_kv):
                for kind in range(2):
                    out[kind][starts[s]: starts[s] + r, h] = _exact_held(st, s, h, p + r, kind)[p:]
        return {"k": out[0], "v": out[1]}
    out = torch.empty(sum(rows), n_kv * G, D, dtype=torch.float64, device="cuda")
    for s, (p, r) in enumerate(zip(pos0, rows)):
        q = st["q"][starts[s]: starts[s] + r].double().view(r, n_kv * G, D)
        hidden = torch.arange(p + r, device="cuda")[None, :] > torch.arange(p, p + r, device="cuda")[:, None]
        for h in range(n_kv):
            k, v = (_exact_held(st, s, h, p + r, kind) for kind in range(2))
            for j in range(h * G, (h + 1) * G):
                score = (q[:, j] @ k.T / math.sqrt(D)).masked_fill(hidden, float("-inf"))
                out[starts[s]: starts[s] + r, j] = torch.softmax(score, -1) @ v
    return out.view(sum(rows), n_kv * G * D)
