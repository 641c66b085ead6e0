"""Plain numpy fp64 definitions of the operators of a loop with several continuations per
prompt: full attention over a 16-bit paged cache, beam selection, rows in a new order.
Literal and slow; shares no code with the CUDA path."""
import math

import numpy as np

BLOCK = 128


def blocks(n):
    return -(-int(n) // BLOCK)


def row_tokens(cache, table, b, h, L):
    """The held rows [n, 128] of head h of the first L tokens of row b; pages that are none have no keys."""
    out = []
    for c in range(blocks(L)):
        pg = table[b, c]
        if 0 <= pg < len(cache):
            out.append(cache[pg, h][:min(BLOCK, L - c * BLOCK)])
    return np.concatenate(out) if out else np.zeros((0, cache.shape[-1]))


def attend(q, kc, vc, table, lens, scale):
    """q [B, Hq, 128], caches [P, Hkv, 128, 128] -> (o, lse) of every row by itself."""
    B, Hq, D = q.shape
    G = Hq // kc.shape[1]
    o, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    for b in range(B):
        L = lens[b] if 0 <= lens[b] <= table.shape[1] * BLOCK else 0
        for h in range(kc.shape[1]):
            K, V = row_tokens(kc, table, b, h, L), row_tokens(vc, table, b, h, L)
            if len(K) == 0:
                continue
            z = q[b, h * G:(h + 1) * G] @ K.T * scale
            top = z.max(-1, keepdims=True)
            p = np.exp(z - top)
            s = p.sum(-1, keepdims=True)
            o[b, h * G:(h + 1) * G] = p @ V / s
            lse[b, h * G:(h + 1) * G] = (top + np.log(s))[:, 0]
    return o, lse


def beam_scores(logits, scores, finished=None, pad=0):
    """Scores [R, V] of all continuations, -inf where there is none."""
    x = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    x = np.minimum(x, 2.0 ** 28)
    out = np.full(x.shape, -np.inf)
    for r in range(len(x)):
        s = float(scores[r])
        if not s > -math.inf:
            continue
        if finished is not None and finished[r]:
            out[r, pad] = s
            continue
        top = x[r].max()
        if top == -math.inf:
            continue
        y = x[r]
        if top < -2.0 ** 28:
            y = np.where(y > -math.inf, np.maximum(y, -2.0 ** 28), y)
            top = y.max()
        out[r] = s + (y - (top + math.log(np.exp(y - top).sum())))
    return out


def beam_select(logits, scores, W, K, finished=None, pad=0):
    """(scores [N, K], parents, tokens), best first, ties to the lower beam and token."""
    all_scores = beam_scores(logits, scores, finished, pad)
    R, V = all_scores.shape
    N = R // W
    so, po, to = np.full((N, K), -np.inf), np.full((N, K), -1), np.full((N, K), -1)
    for n in range(N):
        flat = all_scores[n * W:(n + 1) * W].ravel()
        order = np.argsort(-flat, kind="stable")[:K]
        order = order[flat[order] > -np.inf]
        k = len(order)
        so[n, :k], po[n, :k], to[n, :k] = flat[order], n * W + order // V, order % V
    return so, po, to


def beam_order(logits, scores, W, K, finished=None, pad=0):
    """(parents, tokens) by score, equal ones by the lower beam, then the larger logit, then the lower token:
    beam_select wherever different logits of a beam have different 64-bit scores."""
    all_scores = beam_scores(logits, scores, finished, pad)
    R, V = all_scores.shape
    x = np.minimum(np.where(np.isnan(logits), -np.inf, logits), 2.0 ** 28)
    x[x.max(-1) < -2.0 ** 28] = 0.0
    po, to = np.full((R // W, K), -1), np.full((R // W, K), -1)
    for n in range(R // W):
        rows = slice(n * W, (n + 1) * W)
        w, v = np.divmod(np.arange(W * V), V)
        flat = all_scores[rows].ravel()
        order = np.lexsort((v, -x[rows].ravel(), w, -flat))[:K]
        order = order[flat[order] > -np.inf]
        po[n, :len(order)], to[n, :len(order)] = n * W + w[order], v[order]
    return po, to


def reorder(parents, table, lens, ref):
    """(table, lens, ref, kept) after the call, from copies."""
    t, n, r = table.copy(), lens.copy(), ref.copy()
    B, maxp = table.shape
    good = [0 <= x <= maxp * BLOCK for x in lens]
    kept = np.zeros(B, np.int64)
    for b in range(B):
        p = parents[b]
        if p < -1 or p >= B or (p >= 0 and not good[p]):
            kept[b] = -1
            continue
        kept[b] = 0 if p < 0 else lens[p]
        if p == b:
            continue
        if good[b]:
            for j in range(blocks(lens[b])):
                r[table[b, j]] -= 1
                t[b, j] = -1
        if p >= 0:
            for j in range(blocks(lens[p])):
                t[b, j] = table[p, j]
                r[table[p, j]] += 1
        n[b] = kept[b]
    return t, n, r, kept
