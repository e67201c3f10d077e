"""A paged key/value cache in 64 bits, written from the definitions: row i of
sequence b's n new tokens stands at position length - n + i, and position p lives
in slot p mod page_size of page pages[b][p / page_size].

Test infrastructure only (see the package docstring).
"""
import numpy as np

from .rotary import rotate


def _slots(pages, first, end, page_size):
    p = np.arange(first, end)
    return np.asarray(pages)[p // page_size], p % page_size


def cache_append(q, k, v, k_cache, v_cache, turns, magnitude, interleaved, starts, lengths, pages):
    """(q_out, k_cache, v_cache) after the append, in 64 bits; q [T,H,d], k, v
    [T,H_kv,d], caches [n_pages, page_size, H_kv, d]. Rows of no sequence keep q."""
    q, k, v, kc, vc = (np.array(x, dtype=np.float64) for x in (q, k, v, k_cache, v_cache))
    for b in range(len(lengths)):
        s, e = starts[b], starts[b + 1]
        if e == s:
            continue
        pos = np.arange(lengths[b] - (e - s), lengths[b])

        def turned(x):
            return rotate(x[s:e].transpose(1, 0, 2)[None], turns, pos[None], magnitude,
                          interleaved)[0].transpose(1, 0, 2)

        at = _slots(pages[b], pos[0], lengths[b], kc.shape[1])
        q[s:e], kc[at], vc[at] = turned(q), turned(k), v[s:e]
    return q, kc, vc


def cache_attention(q, k_cache, v_cache, starts, lengths, pages, scale, causal=True, softcap=0.0,
                    left=-1, sinks=0):
    """(O [T,H,d], LSE [T,H], A, X): A = sum of P |v|, which bounds what an error
    of P costs O, and X [T,H] the largest sum of |q| |k| of a visible key."""
    q = np.asarray(q, dtype=np.float64)
    T, H, d = q.shape
    H_kv, page_size = k_cache.shape[2], k_cache.shape[1]
    O, A = np.zeros((T, H, d)), np.zeros((T, H, d))
    LSE, X = np.full((T, H), -np.inf), np.zeros((T, H))
    for b in range(len(lengths)):
        for t in range(starts[b], starts[b + 1]):
            p = lengths[b] - starts[b + 1] + t
            j = np.arange(lengths[b])
            seen = j <= p if causal else j >= 0
            if left >= 0:
                seen &= (j >= p - left) | (j < sinks)
            j = j[seen]
            if len(j) == 0:
                continue
            at = np.asarray(pages[b])[j // page_size], j % page_size
            k, v = (np.asarray(x[at], dtype=np.float64) for x in (k_cache, v_cache))
            for h in range(H):
                g = h // (H // H_kv)
                z = scale * (k[:, g] @ q[t, h])
                if softcap > 0:
                    z = softcap * np.tanh(z / softcap)
                m = z.max()
                w = np.exp(z - m)
                LSE[t, h] = m + np.log(w.sum())
                w /= w.sum()
                O[t, h], A[t, h] = w @ v[:, g], w @ np.abs(v[:, g])
                X[t, h] = scale * (np.abs(k[:, g]) @ np.abs(q[t, h])).max()
    return O, LSE, A, X
