"""Attention side of a serving step, plain -- TEST INFRASTRUCTURE ONLY.

Per-head RMS norms with the position rotation, attention over a paged NVFP4
key/value cache, and the operations on its pages, written from their
definitions (include/moe_gb300.h) in numpy: loops over tokens, heads and pages,
fp64 wherever a result is a rounded real number, and IEEE fp32 step by step
where the definition fixes every rounding (norms and rotation).  Shares no code
with the CUDA path.
"""
from __future__ import annotations

import numpy as np

from . import nvfp4

F32 = np.float32


# ------------------------------------------------------------ norms, rotation
def tree_sum(x: np.ndarray) -> np.ndarray:
    """fp32 sum over the last axis (a power of two): neighbours first."""
    x = np.asarray(x, F32)
    while x.shape[-1] > 1:
        x = (x[..., 0::2] + x[..., 1::2]).astype(F32)
    return x[..., 0]


def rope_pairs(D: int, rot: int, interleaved: bool):
    """The two elements of each rotated pair."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def norm_rope(x, w, eps, cos, sin, interleaved: bool) -> np.ndarray:
    """x fp32 [T, heads, D], w fp32 [D] or None, cos / sin fp32 [T, rot/2]: each
    operation rounded to fp32."""
    x = np.asarray(x, F32)
    D = x.shape[-1]
    if w is not None:
        ms = (tree_sum(x * x) * F32(1.0 / D)).astype(F32) + F32(eps)
        r = (F32(1.0) / np.sqrt(ms, dtype=F32)).astype(F32)
        x = ((x * r[..., None]).astype(F32) * np.asarray(w, F32)).astype(F32)
    rot = 2 * cos.shape[-1]
    if rot:
        a, b = rope_pairs(D, rot, interleaved)
        c, s = cos[:, None, :].astype(F32), sin[:, None, :].astype(F32)
        xa, xb = x[..., a], x[..., b]
        y = x.copy()
        y[..., a] = (xa * c).astype(F32) - (xb * s).astype(F32)
        y[..., b] = (xb * c).astype(F32) + (xa * s).astype(F32)
        x = y
    return x


def norm_rope_f64(x, w, eps, cos, sin, interleaved: bool) -> np.ndarray:
    """The same in fp64, the rotation as a product of complex numbers."""
    x = np.asarray(x, np.float64)
    if w is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    rot = 2 * cos.shape[-1]
    if rot:
        a, b = rope_pairs(x.shape[-1], rot, interleaved)
        z = (x[..., a] + 1j * x[..., b]) * (cos.astype(np.float64) + 1j * sin.astype(np.float64))[:, None, :]
        x = x.copy()
        x[..., a], x[..., b] = z.real, z.imag
    return x


# ----------------------------------------------------------------- the records
def record_bytes(P: int, D: int) -> int:
    return P * D * 9 // 8


def sections(record: np.ndarray, P: int, D: int):
    """A record's bytes as views: key codes [P, D/2], key scales [P, D/16], value codes, value scales."""
    a, b = P * D // 2, P * D // 16
    cut = np.cumsum([a, b, a])
    kc, ks, vc, vs = np.split(record, cut)
    return kc.reshape(P, -1), ks.reshape(P, -1), vc.reshape(P, -1), vs.reshape(P, -1)


def write_token(pool: np.ndarray, slot: int, k: np.ndarray, v: np.ndarray, g_k, g_v, P: int) -> None:
    """k, v fp32 [Hkv, D] into token slot of pool uint8 [num_pages, Hkv, record]."""
    page, off = divmod(int(slot), P)
    for h in range(k.shape[0]):
        kc, ks, vc, vs = sections(pool[page, h], P, k.shape[1])
        q, s, _ = nvfp4.quantize(k[h:h + 1], g_k[h])
        kc[off], ks[off] = q[0], s[0]
        q, s, _ = nvfp4.quantize(v[h:h + 1], g_v[h])
        vc[off], vs[off] = q[0], s[0]


def read_head(pool: np.ndarray, pages, h: int, n: int, D: int, P: int, g_k, g_v):
    """The first n keys and values (fp64 [n, D]) of a sequence's kv head."""
    ks, vs = [], []
    for j in range((n + P - 1) // P):
        kc, ksf, vc, vsf = sections(pool[pages[j], h], P, D)
        m = min(P, n - j * P)
        ks.append(nvfp4.dequantize(kc[:m], ksf[:m], g_k[h]))
        vs.append(nvfp4.dequantize(vc[:m], vsf[:m], g_v[h]))
    if not ks:
        return np.zeros((0, D)), np.zeros((0, D))
    return np.concatenate(ks), np.concatenate(vs)


# ------------------------------------------------------------------- attention
def attention(q, pool, g_k, g_v, q_offsets, kv_lens, table, scale, P: int, causal=True, window=0):
    """q [T, Hq, D] -> (out fp64 [T, Hq, D], lse fp64 [T, Hq], weight and all_v
    fp64 [T, Hq, D]: sum_j p_j |v_j| and sum_j |v_j| / sum_j exp(z_j - max z),
    the scales of the output's relative and absolute rounding errors)."""
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    Hkv = pool.shape[1]
    G = Hq // Hkv
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    weight, all_v = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    for b in range(len(kv_lens)):
        t0, t1, n = int(q_offsets[b]), int(q_offsets[b + 1]), int(kv_lens[b])
        for h in range(Hkv if t1 > t0 else 0):
            K, V = read_head(pool, table[b], h, n, D, P, g_k, g_v)
            key = np.arange(n)
            for t in range(t0, t1):
                place = n - (t1 - t0) + (t - t0)
                see = np.ones(n, bool)
                if causal:
                    see &= key <= place
                if window > 0:
                    see &= key > place - window
                if not see.any():
                    continue
                z = scale * (q[t, h * G:(h + 1) * G] @ K[see].T)
                m = z.max(1, keepdims=True)
                e = np.exp(z - m)
                l = e.sum(1, keepdims=True)
                out[t, h * G:(h + 1) * G] = (e / l) @ V[see]
                weight[t, h * G:(h + 1) * G] = (e / l) @ np.abs(V[see])
                all_v[t, h * G:(h + 1) * G] = np.abs(V[see]).sum(0) / l
                lse[t, h * G:(h + 1) * G] = (m + np.log(l))[:, 0]
    return out, lse, weight, all_v


# ----------------------------------------------------------------------- pages
class Pages:
    """Tables, lengths and counts as plain lists; every operation as one would
    do it by hand, taking the lowest free page."""

    def __init__(self, table, lens, refs, P: int):
        self.table = [list(map(int, r)) for r in table]
        self.lens = list(map(int, lens))
        self.refs = list(map(int, refs))
        self.P = P
        self.M = len(self.table[0]) if self.table else 0

    def used(self, n: int) -> int:
        return -(-n // self.P)

    def free_pages(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def extend(self, counts):
        """counts[row] new tokens; returns (slots, pos) of all tokens in order and the rows that failed."""
        free, slots, pos, failed = self.free_pages(), [], [], []
        taken = 0  # ids are handed out in order of rows, also to rows that then fail
        for r, n in enumerate(counts):
            have, want = self.used(self.lens[r]), self.used(self.lens[r] + n)
            more = max(0, want - have) if n else 0
            fits = want <= self.M
            ids = free[taken:taken + more] if fits else []
            ok = fits and len(ids) == more
            taken += more if fits else 0
            if n and not ok:
                failed.append(r)
            if ok and n:
                for i, p in enumerate(ids):
                    self.table[r][have + i] = p
                    self.refs[p] = 1
            for i in range(n):
                at = self.lens[r] + i
                slots.append(self.table[r][at // self.P] * self.P + at % self.P if ok else -1)
                pos.append(at)
            if ok:
                self.lens[r] += n
        return slots, pos, failed

    def fork(self, src, dst):
        """Returns the (from, to) pairs of pages to copy."""
        free, copies = self.free_pages(), []
        lens, table = list(self.lens), [list(r) for r in self.table]
        for s, d in zip(src, dst):
            n = lens[s]
            full, part = n // self.P, n % self.P
            row = [table[s][j] if j < full else -1 for j in range(self.M)]
            for j in range(full):
                self.refs[table[s][j]] += 1
            if part:
                if free:
                    row[full] = free.pop(0)
                    self.refs[row[full]] = 1
                    copies.append((table[s][full], row[full]))
                else:
                    n = full * self.P
            self.table[d], self.lens[d] = row, n
        return copies

    def free(self, rows):
        for r in dict.fromkeys(rows):
            for j in range(self.used(self.lens[r])):
                self.refs[self.table[r][j]] -= 1
            self.table[r], self.lens[r] = [-1] * self.M, 0

    def compact(self):
        """Returns (remap, pairs of pages to move)."""
        live = [p for p, r in enumerate(self.refs) if r > 0]
        n = len(live)
        holes = [p for p in range(n) if self.refs[p] == 0]
        high = [p for p in live if p >= n]
        remap = [p if r > 0 else -1 for p, r in enumerate(self.refs)]
        for a, b in zip(high, holes):
            remap[a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.table = [[remap[p] if p >= 0 else -1 for p in row] for row in self.table]
        return remap, list(zip(high, holes))
