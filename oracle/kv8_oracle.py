"""CPU oracle of the cache with 8-bit history: one request, tokens one by one,
in 64 bits, from the definitions in include/oscar.h (test infrastructure only)."""
from __future__ import annotations

import numpy as np

D, SINK, RING, BLK, PAGE = 128, 64, 256, 16, 64
QMAX = {0: 448.0, 1: 127.0}
HEAD_BYTES = 4 * 4096 + 32
TINY = 2.0 ** -100


def e4m3_table():
    """Value of every e4m3 byte (S EEEE MMM, bias 7, no infinities, 0x7f NaN)."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(float) - 10))
    v[(b & 127) == 127] = np.nan
    return np.where(b >= 128, -v, v)


E4M3 = e4m3_table()


def encode(y, kind):
    """Nearest code of y (float64, |y| <= qmax), ties to even, as bytes."""
    if kind == 1:
        return np.rint(y).astype(np.int8).view(np.uint8)
    pos = E4M3[:127]  # 0 .. 448, ascending; an even byte has an even significand
    a = np.abs(y)
    i = np.clip(np.searchsorted(pos, a, side="right") - 1, 0, 125)
    mid = (pos[i] + pos[i + 1]) / 2
    up = (a > mid) | ((a == mid) & (i % 2 == 1))
    return ((i + up) | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def decode(codes, kind):
    return E4M3[codes] if kind == 0 else codes.view(np.int8).astype(np.float64)


def quantise(x, kind):
    """x [16][128] -> (bytes [16][128], fp32 scale)."""
    x = x.astype(np.float64)
    if not np.isfinite(x).all():
        return np.zeros(x.shape, np.uint8), np.float32(np.nan)
    am = max(np.abs(x).max(), TINY)
    return encode(x * QMAX[kind] / am, kind), np.float32(np.float32(am) / np.float32(QMAX[kind]))


_i = np.arange(2048)
_c, _g, _q, _b = _i // 512, _i // 64 % 8, _i // 16 % 4, _i % 16
_s, _h, _r, _l = _b // 8, _b // 4 % 2, _b // 2 % 2, _b % 2
PLACE = [(8 * _r + _g) * D + 32 * _c + 8 * _q + 4 * _s + 2 * _h + _l,   # K: token * 128 + channel of each byte
         (8 * _h + 2 * _q + _l) * D + 16 * _g + 4 * _c + 2 * _s + _r]  # V


def pack(codes, side):
    """[16][128] bytes in token order -> the 2048 bytes of a block."""
    return codes.reshape(-1)[PLACE[side]]


def unpack(raw, side):
    out = np.empty(2048, np.uint8)
    out[PLACE[side]] = raw
    return out.reshape(BLK, D)


class Request:
    """One request of Hkv heads.  Tokens are float64 [Hkv][128]."""

    def __init__(self, Hkv, kind):
        self.Hkv, self.kind = Hkv, kind
        self.sink, self.window = [], []   # [(k, v)]
        self.blocks = [[] for _ in range(Hkv)]  # per head: (kcodes, ks, vcodes, vs) in slot order
        self.w_ring = np.zeros((Hkv, 16))
        self.w_hist = [[] for _ in range(Hkv)]

    @property
    def H(self):
        return BLK * len(self.blocks[0])

    @property
    def L(self):
        return len(self.sink) + self.H + len(self.window)

    def append(self, k, v):
        if len(self.sink) < SINK:
            self.sink.append((k, v))
            return
        if len(self.window) == RING:
            old, self.window = self.window[:BLK], self.window[BLK:]
            slot = (self.H // BLK) % 16
            for h in range(self.Hkv):
                kc, ks = quantise(np.stack([t[0][h] for t in old]), self.kind)
                vc, vs = quantise(np.stack([t[1][h] for t in old]), self.kind)
                self.blocks[h].append((kc, ks, vc, vs))
                self.w_hist[h].append(self.w_ring[h, slot])
        at = self.H + len(self.window)
        if at % BLK == 0:
            self.w_ring[:, at // BLK % 16] = 0.0
        self.window.append((k, v))

    def tokens(self, h):
        """(K, V) [L][128] of a head: sink, history, window."""
        out = []
        for side in (0, 1):
            hist = [decode(b[2 * side], self.kind) * np.float64(b[2 * side + 1]) for b in self.blocks[h]]
            rows = ([t[side][h] for t in self.sink], hist, [t[side][h] for t in self.window])
            out.append(np.concatenate([np.asarray(x, np.float64).reshape(-1, D) for x in rows]))
        return out

    def attend(self, q, decay=None):
        """q [Hkv][G][128] -> (out, lse, p [Hkv][G][L]); with decay the weights are updated."""
        G = q.shape[1]
        out, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
        ps = np.zeros((self.Hkv, G, self.L))
        if self.L == 0:
            return out, lse, ps
        with np.errstate(invalid="ignore"):
            for h in range(self.Hkv):
                K, V = self.tokens(h)
                z = q[h].astype(np.float64) @ K.T / np.sqrt(D)
                m = z.max(1, keepdims=True)
                e = np.exp(z - m)
                ps[h] = e / e.sum(1, keepdims=True)
                out[h], lse[h] = ps[h] @ V, m[:, 0] + np.log(e.sum(1))
                if decay is not None:
                    t = ps[h].sum(0)
                    n = self.H // BLK
                    hist = t[len(self.sink):len(self.sink) + self.H].reshape(n, BLK).sum(1)
                    self.w_hist[h] = list(np.asarray(self.w_hist[h]) * decay + hist)
                    win = t[len(self.sink) + self.H:]
                    for j in range(0, len(win), BLK):
                        slot = (n + j // BLK) % 16
                        self.w_ring[h, slot] = self.w_ring[h, slot] * decay + win[j:j + BLK].sum()
        return out, lse, ps

    def evict(self, budget, weights):
        """weights [Hkv][blocks]: the fp32 values that decide."""
        e = max(self.H - budget, 0) // RING * 16
        if not e:
            return
        for h in range(self.Hkv):
            n = len(self.blocks[h])
            w = np.asarray(weights[h][:n], np.float32)
            order = sorted(range(n), key=lambda i: (np.isnan(w[i]), 0.0 if np.isnan(w[i]) else float(w[i]), i))
            gone, keep = set(order[:e]), n - e
            holes = [i for i in range(keep) if i in gone]
            ends = [i for i in range(keep, n) if i not in gone]
            for a, b in zip(holes, ends):
                self.blocks[h][a] = self.blocks[h][b]
                self.w_hist[h][a] = self.w_hist[h][b]
            self.blocks[h] = self.blocks[h][:keep]
            self.w_hist[h] = self.w_hist[h][:keep]
