"""Plain 64-bit restatement of the 4-bit key/value cache for the tests: the pool's bytes, the
block bookkeeping, norms with rotation, and attention.  Shares no code with the library."""
import numpy as np


def code_byte(D, key, col):
    """Byte of a tile's K codes that holds column col of token key (V's codes: + 8 D)."""
    x = {256: key & 7, 128: (key >> 1) & 3, 64: (key >> 2) & 1}[D]
    return key * (D // 2) + (((col // 32) ^ x) * 16) + (col % 32) // 2


def read_slots(pool, slots, kv_heads, P, D):
    """K, V float64 [len(slots), kv_heads, D] of the pool's bytes (uint8 [blocks, bytes])."""
    flat = pool.reshape(-1)
    G = D // 64
    slots = np.asarray(slots, dtype=np.int64)
    heads = np.arange(kv_heads)
    key = slots % 16
    tile = (((slots // P)[:, None] * kv_heads + heads) * (P // 16) + (slots % P // 16)[:, None])
    base = tile * (18 * D)  # [n, K]
    col = np.arange(D)
    byte = np.stack([code_byte(D, k, col) for k in range(16)])[key]  # [n, D]
    out = []
    for which in (0, 1):
        at = base[:, :, None] + which * 8 * D + byte[:, None, :]
        code = (flat[at] >> (4 * (col & 1)).astype(np.uint8)) & 15
        meta = []
        for part in (0, 1):  # scale, bias
            g = np.arange(G)
            if which == 0:
                i = part * 16 * G + key[:, None] * G + g
            else:
                i = 32 * G + part * 16 * G + g * 16 + key[:, None]
            b = base[:, :, None] + 16 * D + 2 * i[:, None, :]
            half = np.stack([flat[b], flat[b + 1]], -1).astype(np.uint8).view(np.float16)[..., 0]
            meta.append(np.repeat(half.astype(np.float64), 64, axis=-1))
        out.append(code * meta[0] + meta[1])
    return out


def norm_rotate(x, w, eps, angles, positions, rot, adjacent, pair_axis):
    """x float64 [T, h, D]; angles [max_pos, rot]; positions [axes, T]."""
    if w is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * w.astype(np.float64)
    y = x.copy()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + rot // 2)
        p = positions[pair_axis[i] if pair_axis else 0]
        c = angles[p, i].astype(np.float64)[:, None]
        s = angles[p, i + rot // 2].astype(np.float64)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


class Tables:
    """The block bookkeeping, one block at a time."""

    def __init__(self, rows, width, blocks, P):
        self.P, self.width, self.blocks = P, width, blocks
        self.table = np.full((rows, width), -1, np.int64)
        self.len = np.zeros(rows, np.int64)
        self.free = list(range(blocks - 1, -1, -1))

    def plan(self, new, max_tokens):
        """(refused, q_start, kv_len, slot, pos)"""
        P, back = self.P, []
        kept = [max(0, int(length) + min(int(n), 0)) for length, n in zip(self.len, new)]
        for b, k in enumerate(kept):
            for j in range(-(-k // P), -(-int(self.len[b]) // P)):
                back.append(int(self.table[b, j]))
                self.table[b, j] = -1
            self.len[b] = k
        self.free += back[::-1]
        add = [max(int(n), 0) for n in new]
        need = sum(-(-(k + a) // P) - -(-k // P) for k, a in zip(kept, add))
        refused = (any(k + a > self.width * P for k, a in zip(kept, add))
                   or need > len(self.free) or sum(add) > max_tokens)
        if refused:
            add = [0] * len(add)
        slot, pos, start = np.full(max_tokens, -1), np.zeros(max_tokens, int), [0]
        for b, (k, a) in enumerate(zip(kept, add)):
            for j in range(-(-k // P), -(-(k + a) // P)):
                self.table[b, j] = self.free.pop()
            for i in range(a):
                pos[start[-1] + i] = k + i
                slot[start[-1] + i] = self.table[b, (k + i) // P] * P + (k + i) % P
            start.append(start[-1] + a)
            self.len[b] = k + a
        return refused, np.array(start), self.len[: len(add)].copy(), slot, pos


def attention(q, k, v, scale, first):
    """q float64 [n, H, D], k and v [L, K, D]: token i sees keys 0 .. first + i."""
    n, H, D = q.shape
    r = H // k.shape[1]
    out = np.zeros((n, H, D))
    for h in range(H):
        x = q[:, h] @ k[:, h // r].T * scale
        x = np.where(np.arange(len(k))[None] > first + np.arange(n)[:, None], -np.inf, x)
        p = np.exp(x - x.max(-1, keepdims=True))
        out[:, h] = (p / p.sum(-1, keepdims=True)) @ v[:, h // r]
    return out


def attention_bound(q, k, v, scale, out):
    """How far a result may be from `out` ([n, H, D]) element by element.

    The output's rounding to bf16 is half a step, 2^-8 |o|.  A weight that enters the second
    product in fp16 is off by 2^-11 of itself, once for itself and once for its product with
    a value's scale; so is a value formed in fp16: three roundings, and a fourth for the fp32
    sums (2^-24 of the same terms per addition, below 2^-11 for the lengths here).  They act on
    scale * code and on the bias, each at most twice the group's largest |v|.  A key formed in
    fp16 moves a score by the sum of D independent roundings of at most 2^-11 |q k| each,
    uniform, so with a spread of scale * sqrt(sum (q k)^2) 2^-11 / sqrt(3); eight times that is
    never passed, and the weight moves by as much of itself (its norm by as much again)."""
    n, H, D = q.shape
    r = H // k.shape[1]
    tol = np.abs(out) * 2.0 ** -8
    for h in range(H):
        kk, vv = k[:, h // r], np.abs(v[:, h // r])
        big = vv.reshape(len(vv), -1, 64).max((0, 2)).repeat(64)[None]  # [1, D]
        spread = scale * np.sqrt((q[:, h] ** 2) @ (kk ** 2).T).max(1, keepdims=True) * 2.0 ** -11
        tol[:, h] += 2 * big * (4 * 2.0 ** -11 + 2 * 8 * spread / np.sqrt(3)) + 1e-6
    return tol


# of the whole output, in the 2-norm: every element's rounding is below 2^-8 of itself, and the
# weights' roundings (2^-11 each, on terms of up to a few times the result) below half of that
ATTENTION_REL = 2.0 ** -8 + 2.0 ** -9
