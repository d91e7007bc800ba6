"""The 4-bit cache restated in numpy, from include/tfl.h: the quantisation formula in
fp32 (whose codes the library must reproduce), the byte layout, and attention in
float64 with a bound on what the library's fp32 / fp16 arithmetic may add."""
import numpy as np

D, GROUP, PAGE, BLOCK, TILE = 128, 64, 128, 16, 18432
HALF = BLOCK * (D // 2 + 8)


def bf16_bits(x):
    """Nearest-even bf16 bit patterns of float32 numbers (finite or not)."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def from_bits(b):
    return (np.asarray(b, np.uint16).astype(np.uint32) << 16).view(np.float32)


def quantise(x):
    """x float32 [..., 128] (bf16 numbers) -> codes uint8 [..., 128], scale and zero float32 [..., 2]."""
    g = np.asarray(x, np.float32).reshape(*x.shape[:-1], D // GROUP, GROUP)
    with np.errstate(all="ignore"):
        zero, high = g.min(-1), g.max(-1)
        span = high - zero
        bad = ~np.isfinite(span)
        scale = from_bits(bf16_bits(span / np.float32(15)))
        n = np.rint((g - zero[..., None]) / np.where(scale > 0, scale, np.float32(1))[..., None])
        n = np.where(((scale > 0) & ~bad)[..., None], np.clip(n, 0, 15), 0)
    n = np.where(np.isnan(n), 0, n).astype(np.uint8).reshape(x.shape)
    return n, np.where(bad, np.float32(0), scale), np.where(bad, np.float32(np.nan), zero)


def values(code, scale, zero):
    """What the codes stand for, float64 [..., 128]."""
    g = code.reshape(*code.shape[:-1], D // GROUP, GROUP).astype(np.float64)
    return (zero[..., None].astype(np.float64) + scale[..., None].astype(np.float64) * g).reshape(code.shape)


def row_bytes(code, pos):
    """The 64 bytes of a row of codes [128] at position pos."""
    out = np.zeros(64, np.uint8)
    for c in range(8):
        at = 8 * (c ^ (4 if pos & 2 else 0))
        for j in range(2):
            n = code[64 * j + 8 * c: 64 * j + 8 * c + 8]
            out[at + 4 * j: at + 4 * j + 4] = n[0::2] | (n[1::2] << 4)
    return out


class Cache:
    """A cache's bytes on the host; table: logical -> physical page (identity by default)."""

    def __init__(self, layers, n_kv, max_positions, fill=0, table=None):
        self.layers, self.n_kv = layers, n_kv
        self.pages = (max_positions + PAGE - 1) // PAGE
        self.table = np.arange(self.pages, dtype=np.int32) if table is None else np.asarray(table, np.int32)
        self.table_bytes = (self.pages * 4 + 255) // 256 * 256
        self.bytes = np.full(self.table_bytes + layers * self.pages * n_kv * TILE, fill, np.uint8)
        self.bytes[: self.pages * 4] = self.table.view(np.uint8)

    def places(self, layer, pos, head, kind):
        """(byte of the row's codes, byte of its scales) in the buffer."""
        tile = (layer * self.pages + int(self.table[pos // PAGE])) * self.n_kv + head
        half = self.table_bytes + tile * TILE + pos % PAGE // BLOCK * 2 * HALF + kind * HALF
        return half + pos % BLOCK * 64, half + BLOCK * 64 + pos % BLOCK * 8

    def put(self, layer, pos, kind, code, scale, zero):
        """One position's codes [n_kv, 128], scale and zero [n_kv, 2]."""
        for h in range(self.n_kv):
            at, meta = self.places(layer, pos, h, kind)
            self.bytes[at: at + 64] = row_bytes(code[h], pos)
            m = np.stack([bf16_bits(scale[h]), np.where(np.isnan(zero[h]), np.uint16(0x7FC0), bf16_bits(zero[h]))], -1)
            self.bytes[meta: meta + 8] = np.ascontiguousarray(m, np.uint16).view(np.uint8).reshape(-1)

    def get(self, layer, n, kind):
        """(code, scale, zero) of positions 0..n-1: [n, n_kv, ...]."""
        pos = np.arange(n)
        tile = (layer * self.pages + self.table[pos // PAGE].astype(np.int64))[:, None] * self.n_kv + np.arange(self.n_kv)
        half = self.table_bytes + tile * TILE + (pos % PAGE // BLOCK * 2 * HALF + kind * HALF)[:, None]
        rows = self.bytes[(half + (pos % BLOCK * 64)[:, None])[..., None] + np.arange(64)]
        meta = self.bytes[(half + (BLOCK * 64 + pos % BLOCK * 8)[:, None])[..., None] + np.arange(8)]
        meta = from_bits(np.ascontiguousarray(meta).view(np.uint16)).reshape(n, self.n_kv, 2, 2)
        code = np.zeros((n, self.n_kv, D), np.uint8)
        swap = np.where(pos & 2, 4, 0)
        for c in range(8):
            for j in range(2):
                for b in range(4):
                    byte = np.take_along_axis(rows, (8 * (c ^ swap) + 4 * j + b)[:, None, None].repeat(self.n_kv, 1), 2)[..., 0]
                    code[..., 64 * j + 8 * c + 2 * b] = byte & 15
                    code[..., 64 * j + 8 * c + 2 * b + 1] = byte >> 4
        return code, meta[..., 0], meta[..., 1]


def attention(q, pos, kq, vq):
    """q float64 [n_q, 128] of one row at position pos; kq, vq = (code, scale, zero) of
    positions 0..pos.  Returns (out, bound) [n_q, 128] float64: |library - out| <= bound.

    The bound, with P the exact weights (sum 1), V = z + s n:
      2^-8 |out|                       the output's rounding to bf16 (half a step), doubled below for
                                       the rounding's sensitivity to everything else: x (1 + 2^-7)
      2^-11 sum P s n                  each weight times its value scale, rounded once to fp16 (half a step)
      T 2^-30 max(P s n)               such a product in the subnormal range of fp16 (the largest of a warp
                                       is kept at 2^6 or more, the subnormal half step is 2^-25)
      (2 ds + 2^-16) sum P (|z| + s n) fp32: a score error ds moves a weight and the sum it is divided by
                                       by e^ds each; 2^-16 covers 2^x (2^-22), and sums of products in
                                       fp32 in chains of at most 64 steps (64 x 2^-23)
      ds = 2^-18 max_t sum_d |q| (|z| + s n) / sqrt(128)   (128-term fp32 sums: 32 steps x 2^-23)
    """
    n_q = q.shape[0]
    n_kv = kq[0].shape[1]
    g = n_q // n_kv
    out, bound = np.zeros((n_q, D)), np.zeros((n_q, D))
    with np.errstate(all="ignore"):
        for h in range(n_kv):
            part = lambda c: (c[0][: pos + 1, h], c[1][: pos + 1, h], c[2][: pos + 1, h])  # noqa: E731
            kc, ks, kz = part(kq)
            vc, vs, vz = part(vq)
            k, v = values(kc, ks, kz), values(vc, vs, vz)
            zero = np.zeros_like(kz)
            k_abs = np.abs(np.repeat(kz, GROUP, -1)) + values(kc, ks, zero)
            v_sn = values(vc, vs, zero)
            v_abs = np.abs(np.repeat(vz, GROUP, -1).astype(np.float64)) + v_sn
            for j in range(h * g, (h + 1) * g):
                s = k @ q[j] / np.sqrt(D)
                p = np.exp(s - s.max())
                p /= p.sum()
                ds = 2.0 ** -18 * (k_abs @ np.abs(q[j])).max() / np.sqrt(D)
                out[j] = p @ v
                bound[j] = (1 + 2.0 ** -7) * (2.0 ** -8 * np.abs(out[j]) + 2.0 ** -11 * (p @ v_sn)
                                              + (pos + 1) * 2.0 ** -30 * (p[:, None] * v_sn).max(0)
                                              + (2 * ds + 2.0 ** -16) * (p @ v_abs)) + 1e-37
    return out, bound
