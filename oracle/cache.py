"""Ragged attention over the paged cache, rotary appends and the page table (oracle).

TEST INFRASTRUCTURE ONLY -- see the package docstring.

Plain definitions: softmax attention of every query token over the dequantised
visible positions in float64; rotations by angles formed in Python integers
and floats; the page table kept row after row on the host.
"""

import math

import numpy as np

from .attention import LOG2E
from .codecs import dequant_page


def sequence_kv(Hkv, P, pools, page_codec, block_table, b, length):
    """K, V float64 [Hkv][n][D], the positions of those n keys, their pages' V scales
    [Hkv][n] (1 for 16-bit pages) and the number of pages that name no slot (left out)."""
    K, V, pos, vs, bad = [], [], [], [], 0
    for p in range((length + P - 1) // P):
        codec, slot = int(page_codec[b, p]), int(block_table[b, p])
        if codec not in pools or not 0 <= slot < pools[codec][0].shape[0]:
            bad += 1
            continue
        n = min(P, length - p * P)
        codes, meta = pools[codec]
        K.append(np.stack([dequant_page(codec, codes, meta, slot, 0, h)[:n] for h in range(Hkv)]))
        V.append(np.stack([dequant_page(codec, codes, meta, slot, 1, h)[:n] for h in range(Hkv)]))
        pos.append(p * P + np.arange(n))
        vs.append(np.repeat(np.ones(Hkv) if codec < 2 else np.asarray(meta[slot, 1], np.float64), n).reshape(Hkv, n))
    if not K:
        return None, None, np.zeros(0, int), None, bad
    return np.concatenate(K, 1), np.concatenate(V, 1), np.concatenate(pos), np.concatenate(vs, 1), bad


def paged_extend(q, q_start, Hkv, P, pools, page_codec, block_table, seq_lens, scale, causal=True):
    """q float64 [total][Hq][D].  Returns o, lse2, bad and, for error bounds,
    av = sum_j p_j |v_j| and pc = max_j (p_j s_j) sum_j |v_j| / s_j with the V scales s_j
    (as o, over sum_j p_j), qk = max_j scale log2(e) sum_d |q_d k_jd| and
    smax = max_j |score_j| in the log2 domain (as lse2).  Rows of no sequence and rows
    that see nothing have o = 0, lse2 = -inf."""
    total, Hq, D = q.shape
    G = Hq // Hkv
    o, av, pc = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    lse2 = np.full((total, Hq), -math.inf)
    qk, smax = np.zeros((total, Hq)), np.zeros((total, Hq))
    bad = 0
    max_pages = block_table.shape[1]
    for b in range(len(seq_lens)):
        t0, t1 = int(q_start[b]), int(q_start[b + 1])
        if t1 <= t0:
            continue
        L = max(0, min(int(seq_lens[b]), max_pages * P))
        K, V, pos, vs, nbad = sequence_kv(Hkv, P, pools, page_codec, block_table, b, L)
        bad += nbad
        if K is None:
            continue
        for t in range(t0, t1):
            keep = pos <= L - (t1 - t0) + (t - t0) if causal else np.ones(len(pos), bool)
            if not keep.any():
                continue
            for hq in range(Hq):
                k, v = K[hq // G][keep], V[hq // G][keep]
                s = scale * (k @ q[t, hq])
                m = s.max()
                w = np.exp(s - m)
                w_sum = w.sum()
                o[t, hq], av[t, hq] = w @ v / w_sum, w @ np.abs(v) / w_sum
                f = vs[hq // G][keep]
                codes = np.abs(v) / np.where(f > 0, f, 1.0)[:, None]
                pc[t, hq] = (w * f).max() / w_sum * codes.sum(0)
                lse2[t, hq] = (m + math.log(w_sum)) * LOG2E
                qk[t, hq] = scale * LOG2E * (np.abs(k) @ np.abs(q[t, hq])).max()
                smax[t, hq] = np.abs(s).max() * LOG2E
    return o, lse2, bad, av, pc, qk, smax


def rotate(x, positions, inv_freq, pair_axis, adjacent):
    """x float64 [tokens][heads][D]; positions int [n_axes][tokens]; a pair whose
    axis does not exist is not turned.  The turn is reduced exactly: position
    times frequency as a fraction of the frequency's own binary expansion."""
    from fractions import Fraction
    half = len(inv_freq)
    out = np.array(x, np.float64)
    two_pi = Fraction("6.283185307179586476925286766559005768394338798750")
    for i in range(half):
        ax = 0 if pair_axis is None else int(pair_axis[i])
        if ax >= positions.shape[0]:
            continue
        turn = Fraction(float(inv_freq[i])) / two_pi
        frac = [turn * int(p) for p in positions[ax]]
        ang = np.array([float((f - math.floor(f)) * two_pi) for f in frac])
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        xa, xb = np.array(x[..., a], np.float64), np.array(x[..., b], np.float64)
        out[..., a] = xa * c - xb * s
        out[..., b] = xb * c + xa * s
    return out


def append_places(q_start, seq_lens, P, page_codec, block_table, codec, n_slots):
    """Per token: (slot, row), or None where it is not stored; tokens of no sequence
    are absent."""
    places = {}
    for b in range(len(seq_lens)):
        t0, t1 = int(q_start[b]), int(q_start[b + 1])
        for t in range(t0, t1):
            c = int(seq_lens[b]) - (t1 - t0) + (t - t0)
            page = c // P
            ok = c >= 0 and page < block_table.shape[1] and page_codec[b, page] == codec and \
                0 <= block_table[b, page] < n_slots
            places[t] = (int(block_table[b, page]), c % P) if ok else None
    return places


def fork_pages(parents, n_new, new_codec, n_slots, refs, page_codec, block_table, seq_lens, P):
    """n_slots / refs: dict codec -> slots / counts.  Returns the new table, codecs,
    lengths, counts, the page copies [(codec, src, dst)] and the anomaly count."""
    B, max_pages = block_table.shape
    refs = {c: np.array(r, np.int64) for c, r in refs.items()}
    cap, status = max_pages * P, 0

    def named(codec, slot):
        return codec in n_slots and 0 <= slot < n_slots[codec]

    old = []
    for b in range(B):
        if not 0 <= seq_lens[b] <= cap:
            status += 1
        old.append(min(max(int(seq_lens[b]), 0), cap))
    rows, lens, adds = [], [], []
    for b in range(B):
        par = int(parents[b])
        if not -1 <= par < B:
            par = -1
            status += 1
        n = 0 if par < 0 else (old[par] + P - 1) // P
        row = [(int(page_codec[par, j]), int(block_table[par, j])) for j in range(n)]
        status += sum(not named(*e) for e in row)
        if par != b:
            for j in range((old[b] + P - 1) // P):
                e = (int(page_codec[b, j]), int(block_table[b, j]))
                if named(*e):
                    refs[e[0]][e[1]] -= 1
            for e in row:
                if named(*e):
                    refs[e[0]][e[1]] += 1
        add = int(n_new[b]) if par >= 0 and n_new is not None else 0
        if add < 0:
            add, status = 0, status + 1
        length = 0 if par < 0 else old[par]
        if length + add > cap:
            add, status = cap - length, status + 1
        rows.append(row)
        lens.append(length)
        adds.append(add)
    free = {c: [s for s in range(n_slots[c]) if refs[c][s] == 0] for c in n_slots}
    writers = {}
    for b in range(B):
        if adds[b] and lens[b] % P and named(*rows[b][-1]):
            writers.setdefault(rows[b][-1], []).append(b)
    keeps = {w[0] for e, w in writers.items() if refs[e[0]][e[1]] == len(w)}
    writes = {b for w in writers.values() for b in w}
    copies = []

    def take(codec):
        nonlocal status
        if free[codec]:
            s = free[codec].pop(0)
            refs[codec][s] = 1
            return s
        status += 1
        return -1

    for b in range(B):
        if b in writes and b not in keeps:
            codec, src = rows[b][-1]
            dst = take(codec)
            refs[codec][src] -= 1
            rows[b][-1] = (codec, dst)
            if dst >= 0:
                copies.append((codec, src, dst))
        while len(rows[b]) * P < lens[b] + adds[b]:
            rows[b].append((new_codec, take(new_codec)))
    table = np.full((B, max_pages), -1, np.int32)
    codecs = np.zeros((B, max_pages), np.uint8)
    for b, row in enumerate(rows):
        for j, (c, s) in enumerate(row):
            table[b, j], codecs[b, j] = s, c
    return table, codecs, np.array(lens) + np.array(adds), refs, copies, status


def compact_pages(codec, ref, page_codec, block_table, seq_lens, P):
    """Returns the new table, counts, moves [(src, dst)], live slots and anomalies."""
    ref = np.maximum(np.asarray(ref, np.int64), 0)
    live = [s for s in range(len(ref)) if ref[s] > 0]
    moves = list(zip([s for s in live if s >= len(live)], [s for s in range(len(live)) if ref[s] == 0]))
    to = dict(moves)
    out = np.where(np.arange(len(ref)) < len(live), ref, 0)
    for s, d in moves:
        out[d] = ref[s]
    table, bad = np.array(block_table), 0
    for b in range(table.shape[0]):
        for j in range(table.shape[1]):
            if page_codec[b, j] == codec and j * P < seq_lens[b]:
                s = int(table[b, j])
                if not 0 <= s < len(ref):
                    bad += 1
                table[b, j] = to.get(s, s)
    return table, out, moves, len(live), bad
