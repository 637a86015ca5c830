"""Float64 reference of the full-rank cache held in 8 bits (NumPy only).

Shares no code with the CUDA path.  A block is 64 tokens of one (sequence,
KV head, side); it is quantised when its last token arrives, the tokens of
the open block stay as they came.
"""
import numpy as np

BLOCK = 64
LEAST = 2.0 ** -100
TOP = {"int8": 127.0, "e4m3": 448.0}


def e4m3_table() -> np.ndarray:
    """The non-negative e4m3 values in order: exponent field 0 is 2^-6 * m / 8,
    field e is 2^(e - 7) * (1 + m / 8); field 15 with m = 7 is NaN."""
    v = [2.0 ** -6 * m / 8 for m in range(8)]
    for e in range(1, 16):
        v += [2.0 ** (e - 7) * (1 + m / 8) for m in range(8)]
    return np.array(v[:-1])


_TABLE = e4m3_table()


def round_e4m3(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value, ties to the even mantissa (the even table index)."""
    a = np.abs(x)
    hi = np.clip(np.searchsorted(_TABLE, a), 1, len(_TABLE) - 1)
    lo = hi - 1
    dl, dh = a - _TABLE[lo], _TABLE[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.copysign(_TABLE[np.where(up, hi, lo)], x)


def quantise_block(x: np.ndarray, code: str):
    """codes (as the numbers they are) and fp32 scale of one block [64, 128]."""
    x = np.asarray(x, np.float64)
    if not np.all(np.isfinite(x)):
        return np.zeros_like(x), np.float32(np.nan)
    a = max(np.max(np.abs(x)), LEAST)
    y = TOP[code] * x / a
    y = np.rint(y) if code == "int8" else round_e4m3(y)
    return y, np.float32(a) / np.float32(TOP[code])


class QuantCacheOracle:
    def __init__(self, B: int, H: int, code: str):
        self.B, self.H, self.code = B, H, code
        self.rows = [[[np.zeros((0, 128)) for _ in range(2)] for _ in range(H)] for _ in range(B)]

    def length(self, b: int) -> int:
        return self.rows[b][0][0].shape[0]

    def append(self, k, v, n_new=None):
        k, v = np.asarray(k, np.float64), np.asarray(v, np.float64)
        for b in range(self.B):
            n = k.shape[2] if n_new is None else int(np.clip(n_new[b], 0, k.shape[2]))
            for h in range(self.H):
                for side, x in enumerate((k, v)):
                    self.rows[b][h][side] = np.concatenate([self.rows[b][h][side], x[b, h, :n]])

    def truncate(self, b: int, length: int):
        for h in range(self.H):
            for side in range(2):
                self.rows[b][h][side] = self.rows[b][h][side][:length]

    def stored(self, b: int, h: int, side: int):
        """codes [full, 128], scales [full / 64] (fp32) and the open rows."""
        x = self.rows[b][h][side]
        full = x.shape[0] // BLOCK * BLOCK
        codes, scales = np.zeros((full, 128)), np.zeros(full // BLOCK, np.float32)
        for j in range(full // BLOCK):
            codes[j * BLOCK:(j + 1) * BLOCK], scales[j] = quantise_block(
                x[j * BLOCK:(j + 1) * BLOCK], self.code)
        return codes, scales, x[full:]

    def values(self, b: int, h: int, side: int, dtype=np.float64) -> np.ndarray:
        """What the cache holds for (b, h): [tokens, 128]; in float32 the
        product code * scale is rounded once, as a read-back gives it."""
        codes, scales, rest = self.stored(b, h, side)
        y = codes.astype(dtype) * np.repeat(scales.astype(dtype), BLOCK)[:, None]
        return np.concatenate([y, rest.astype(dtype)])

    def attend(self, q, scale: float, n_q=None):
        """o [B, H_q, n, 128] (NaN rows past a sequence's queries) and, for the
        tests' error bounds, w = sum p |v| of the same shape and
        s [B, H_q, n, 4]: a row's largest sum |q k| * scale, its largest
        |score|, its largest p * (largest |v| of the token's block) and the
        largest |v| it sees."""
        q = np.asarray(q, np.float64)
        B, Hq, n, _ = q.shape
        G = Hq // self.H
        o, w = np.full(q.shape, np.nan), np.zeros(q.shape)
        s2 = np.zeros((B, Hq, n, 4))
        for b in range(B):
            L = self.length(b)
            m = n if n_q is None else int(np.clip(n_q[b], 0, n))
            for h in range(self.H):
                K, V = self.values(b, h, 0), self.values(b, h, 1)
                top = np.concatenate([np.full(min(BLOCK, L - j), np.max(np.abs(V[j:j + BLOCK])))
                                      for j in range(0, L, BLOCK)] or [np.zeros(0)])
                for g in range(h * G, h * G + G):
                    for i in range(m):
                        seen = L - m + i + 1
                        if seen <= 0:
                            o[b, g, i] = 0
                            continue
                        s = K[:seen] @ q[b, g, i] * scale
                        p = np.exp(s - np.max(s))
                        p /= p.sum()
                        o[b, g, i] = p @ V[:seen]
                        w[b, g, i] = p @ np.abs(V[:seen])
                        s2[b, g, i] = (np.max(np.abs(K[:seen]) @ np.abs(q[b, g, i])) * scale,
                                       np.max(np.abs(s)), np.max(p * top[:seen]),
                                       np.max(np.abs(V[:seen])))
        return o, w, s2
