"""Plain numpy fp64 definitions of the long-context operators: the prologue for any
rotary layout, the 4-bit cache format, the decode step over it and the page tables.
Literal and slow; shares no code with the CUDA path."""
import math

import numpy as np

BLOCK, TOPK, D = 128, 16, 128
SLAB = 9216
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_value(byte):
    """The number that an e4m3 byte stands for (bias 7, no infinities, 0x7F / 0xFF = NaN)."""
    byte = np.asarray(byte).astype(np.int64)
    e, m = (byte >> 3) & 15, byte & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(byte & 128, -v, v)


E4M3 = e4m3_value(np.arange(127))        # 0 .. 448, ascending


def nearest_even(v, levels):
    """Index of the level nearest to v >= 0; ties to the even index, above the last: the last."""
    hi = np.clip(np.searchsorted(levels, v, side="left"), 1, len(levels) - 1)
    up, down = levels[hi] - v, v - levels[hi - 1]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def bf16_round(x):
    """fp64 -> nearest bf16 value (ties to even), in fp64."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126)))
        ulp = 2.0 ** (e - 7)
        return np.where(np.isfinite(x), np.rint(x / ulp) * ulp, x)


# ------------------------------------------------------------------ rotation

def rope_freqs(dim, base, scaling="none", factor=1.0, orig_len=32768.0, fast=32.0, slow=1.0):
    if scaling == "ntk":
        base = base * factor ** (dim / (dim - 2))
    f = [base ** (-2 * i / dim) for i in range(dim // 2)]
    gain = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "yarn":
        out = []
        for x in f:
            turns = orig_len * x / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - slow) / (fast - slow)))
            out.append(x / factor * (1 - keep) + x * keep)
        f, gain = out, 0.1 * math.log(factor) + 1.0
    return np.array(f), gain


def positions_of(cu, T):
    pos = np.zeros(T, np.int64)
    for a, b in zip(cu[:-1], cu[1:]):
        pos[a:b] = np.arange(b - a)
    return pos


def rotate(z, pos, freqs, gain, layout, back=False):
    """z [T, H, D] with its first 2 len(freqs) channels turned, as complex numbers."""
    R = 2 * len(freqs)
    turn = gain * np.exp((-1j if back else 1j) * pos[:, None].astype(np.float64) * freqs)[:, None]
    y = z.copy()
    a, b = (slice(0, R // 2), slice(R // 2, R)) if layout == "half" else (slice(0, R, 2), slice(1, R, 2))
    t = (z[..., a] + 1j * z[..., b]) * turn
    y[..., a], y[..., b] = t.real, t.imag
    return y


def prologue(x, w, pos, freqs, gain=1.0, layout="half", eps=1e-6):
    z = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1 + w)
    return rotate(z, pos, freqs, gain, layout)


def prologue_bwd(x, dy, w, pos, freqs, gain=1.0, layout="half", eps=1e-6):
    dz = rotate(dy, pos, freqs, gain, layout, back=True)
    if w is None:
        return dz, None
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh, g = x * r, dz * (1 + w)
    return r * (g - xh * (g * xh).mean(-1, keepdims=True)), (dz * xh).sum((0, 1))


# ------------------------------------------------------------------ 4 bits

def quantise(x, gain=1.0):
    """x [..., 128] -> (codes 0 .. 15 [..., 128], scale bytes [..., 8])."""
    b = x.reshape(*x.shape[:-1], 8, 16) / gain
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    # the quotient by 6 is rounded to fp32 before it is rounded to e4m3
    want = (np.abs(b).max(-1).astype(np.float32) / np.float32(6)).astype(np.float64)
    sb = nearest_even(want, E4M3)
    s = E4M3[sb][..., None]
    m = np.abs(b) / np.where(s > 0, s, 1.0)
    code = np.where(s > 0, nearest_even(m, E2M1) + 8 * np.signbit(b), 0)
    return (np.where(bad[..., None], 0, code).reshape(x.shape).astype(np.uint8),
            np.where(bad, 0x7F, sb).astype(np.uint8))


def held(codes, scales, gain=1.0):
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return (v.reshape(*codes.shape[:-1], 8, 16) * e4m3_value(scales)[..., None]).reshape(codes.shape) * gain


def slab_values(slab, gain=1.0):
    """uint8 [..., 9216] -> [..., 128 tokens, 128]"""
    byte = slab[..., :8192].reshape(*slab.shape[:-1], 128, 64)
    codes = np.stack([byte & 15, byte >> 4], -1).reshape(*slab.shape[:-1], 128, 128)
    return held(codes, slab[..., 8192:].reshape(*slab.shape[:-1], 128, 8), gain)


def make_slab(x, gain=1.0):
    """[..., 128 tokens, 128] -> uint8 [..., 9216]"""
    codes, scales = quantise(x, gain)
    byte = (codes[..., 0::2] | (codes[..., 1::2] << 4)).reshape(*x.shape[:-2], 8192)
    return np.concatenate([byte, scales.reshape(*x.shape[:-2], 1024)], -1)


# ------------------------------------------------------------------ decode

def decode_scores(q_idx, kidx, table, b, h, L):
    """Largest index logit of every block of sequence b (kidx: slabs); -inf for bad pages."""
    n = (L + BLOCK - 1) // BLOCK
    out = np.full(n, -np.inf)
    for c in range(n):
        pg = table[b, c]
        if 0 <= pg < kidx.shape[0]:
            k = slab_values(kidx[pg, h])[:min(BLOCK, L - c * BLOCK)]
            out[c] = (k @ q_idx[b, h]).max()
    return out


def select(scores, n_init=0):
    """Own block (the last), the first n_init, the best others (ties: lower id): 16 at most.
    Also the relative gap between the last kept and the first dropped score."""
    own = len(scores) - 1
    first = list(range(min(n_init, own)))
    rest = sorted(range(len(first), own), key=lambda i: (-scores[i], i))
    room = TOPK - 1 - len(first)
    gap = np.inf
    if len(rest) > room > 0:
        a, b = scores[rest[room - 1]], scores[rest[room]]
        gap = abs(a - b) / max(abs(a), abs(b), 1e-300)
    return first + sorted(rest[:room]) + [own], gap


def attend(q, kc, vc, table, b, h, L, sel, scale, k_gain=1.0, v_gain=1.0):
    """q [G, 128] over the keys of the selected blocks."""
    K, V = [], []
    for c in sel:
        pg = table[b, c]
        if 0 <= pg < kc.shape[0]:
            n = min(BLOCK, L - c * BLOCK)
            K.append(slab_values(kc[pg, h], k_gain)[:n])
            V.append(slab_values(vc[pg, h], v_gain)[:n])
    if not K:
        return np.zeros((q.shape[0], D))
    K, V = np.concatenate(K), np.concatenate(V)
    z = q @ K.T * scale
    p = np.exp(z - z.max(-1, keepdims=True))
    return p @ V / p.sum(-1, keepdims=True)


# ------------------------------------------------------------------ pages

class Pages:
    """Tables and page contents (one integer per page stands for its bytes)."""

    def __init__(self, table, lens, ref, content):
        self.table, self.lens, self.ref = table.copy(), lens.copy(), ref.copy()
        self.content = content.copy()

    @staticmethod
    def blocks(n):
        return -(-int(n) // BLOCK)

    def fork(self, src, dst, keep=None):
        before = self.lens.copy()
        out = []
        taken = set()
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < len(before) and 0 <= d < len(before)) or s == d or before[d] != 0 \
                    or d in taken:
                out.append(-1)
                continue
            taken.add(d)
            k = before[s] if keep is None else min(max(keep[i], 0), before[s])
            for j in range(self.blocks(k)):
                self.table[d, j] = self.table[s, j]
                self.ref[self.table[s, j]] += 1
            self.lens[d] = k
            out.append(k)
        return np.array(out)

    def free(self, rows, keep=None):
        before = self.lens.copy()
        out = []
        taken = set()
        for i, r in enumerate(rows):
            k = 0 if keep is None else keep[i]
            if not 0 <= r < len(before) or k < 0:
                out.append(-1)
            elif k >= before[r]:
                out.append(0)
            elif r in taken:
                out.append(-1)
            else:
                taken.add(r)
                for j in range(self.blocks(k), self.blocks(before[r])):
                    self.ref[self.table[r, j]] -= 1
                    self.table[r, j] = -1
                self.lens[r] = k
                out.append(before[r] - k)
        return np.array(out)

    def extend(self, add):
        free = [p for p in range(len(self.ref)) if self.ref[p] == 0]
        shared = self.ref.copy()
        wanted, done = 0, []
        for b, a in enumerate(add):
            L = self.lens[b]
            if a < 0 or L + a > self.table.shape[1] * BLOCK:
                done.append(0)
                continue
            need = self.blocks(L + a) - self.blocks(L)
            cow = a > 0 and L % BLOCK != 0 and shared[self.table[b, L // BLOCK]] > 1
            at, wanted = wanted, wanted + need + cow
            if need + cow > 0 and wanted > len(free):
                done.append(0)
                continue
            got = free[at:wanted]
            if cow:
                old = self.table[b, L // BLOCK]
                self.content[got[0]] = self.content[old]
                self.ref[old] -= 1
                self.table[b, L // BLOCK] = got[0]
            for j in range(need):
                self.table[b, self.blocks(L) + j] = got[j + cow]
            for p in got:
                self.ref[p] = 1
            self.lens[b] = L + a
            done.append(1)
        return np.array(done)

    def compact(self):
        used = [p for p in range(len(self.ref)) if self.ref[p] > 0]
        n = len(used)
        to = {p: p for p in used if p < n}
        to.update(zip([p for p in used if p >= n], [p for p in range(n) if self.ref[p] == 0]))
        ref, content = self.ref.copy(), self.content.copy()
        for p, d in to.items():
            ref[d], content[d] = self.ref[p], self.content[p]
        ref[n:] = 0
        for b, L in enumerate(self.lens):
            for j in range(self.blocks(L)):
                self.table[b, j] = to[self.table[b, j]]
        self.ref, self.content = ref, content
        page_map = np.full(len(ref), -1)
        for p, d in to.items():
            page_map[p] = d
        return page_map, n
