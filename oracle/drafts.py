"""Drafted trees, windows of several tokens, head norms, attention weights and eviction (oracle).

TEST INFRASTRUCTURE ONLY -- see the package docstring.

Plain definitions in float64, one row or position at a time; what is stored in 8 bits
goes through the encoders of codecs.py.
"""

import math

import numpy as np

from .attention import LOG2E
from .cache import sequence_kv
from .codecs import CODEC_BF16, CODEC_FP16, CODEC_FP8_E4M3, CODEC_INT8, dequant_page, f64_to_bf16_bits, quantize_unit_fp8, quantize_unit_int8


def window_sees(window, sinks):
    """paged_extend's rule of sight for a sliding window and first tokens."""
    def sees(b, i, n, L, pos):
        at = L - n + i
        return (pos <= at) & ((pos > at - window) | (pos < sinks))
    return sees


def tree_sees(masks):
    """... for trees: masks[b][i] is an integer whose bit x says that token i sees token x."""
    def sees(b, i, n, L, pos):
        return np.array([p < L - n or (p - (L - n) < n and masks[b][i] >> int(p - (L - n)) & 1 == 1) for p in pos], bool)
    return sees


def head_norm(x, weight, eps):
    """x float64 [...][D]: each row over the root of its mean square, times weight."""
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if weight is None else np.asarray(weight, np.float64))


def accept_tokens(q_start, seq_lens, path, n_path, P, page_codec, block_table, codec, n_slots):
    """Returns the moves [((slot, row), (slot, row))] in order, the new lengths and the anomaly count."""
    moves, lens, bad = [], [], 0

    def place(b, c):
        j = c // P
        if j < block_table.shape[1] and page_codec[b, j] == codec and 0 <= block_table[b, j] < n_slots:
            return int(block_table[b, j]), c % P
        return None

    for b in range(len(seq_lens)):
        L, n = int(seq_lens[b]), max(int(q_start[b + 1]) - int(q_start[b]), 0)
        m = min(max(int(n_path[b]), 0), path.shape[1])
        bad += m != int(n_path[b])
        if L < n:
            bad += 1
            lens.append(L)
            continue
        k, before = 0, -1
        while k < m:
            x = int(path[b, k])
            if not before < x < n:
                bad += 1
                break
            if x != k:
                a, z = place(b, L - n + x), place(b, L - n + k)
                if a is None or z is None:
                    bad += 1
                else:
                    moves.append((a, z))
            before = x
            k += 1
        lens.append(L - n + k)
    return moves, np.array(lens), bad


def attn_weights(q, q_start, lse2, Hkv, P, pools, page_codec, block_table, seq_lens, scale, weights, decay, causal=True):
    """weights float64 [B][Hkv][positions].  Returns the new ones, the bad pages, and for error
    bounds the sum of the added weights times what a score may be off by: per weight
    ln 2 (D 2^-23 scale log2(e) sum_d |q_d k_d| + 2^-22 (|score| + |lse2|)) + 2^-21 (and
    fp32's rounding of the sum)."""
    _, Hq, D = q.shape
    G, cap = Hq // Hkv, block_table.shape[1] * P
    out, err, bad = np.array(weights), np.zeros(weights.shape), 0
    for b in range(len(seq_lens)):
        L = max(0, min(int(seq_lens[b]), cap))
        K, _, pos, _, nbad = sequence_kv(Hkv, P, pools, page_codec, block_table, b, L)
        bad += nbad
        out[b, :, :L] = out[b, :, :L] * decay if decay else 0.0
        t0, t1 = int(q_start[b]), int(q_start[b + 1])
        if K is None:
            continue
        for t in range(t0, t1):
            keep = pos <= L - (t1 - t0) + (t - t0) if causal else np.ones(len(pos), bool)
            for hq in range(Hq):
                if lse2[t, hq] == -math.inf or not keep.any():
                    continue
                k = K[hq // G][keep]
                s = scale * LOG2E * (k @ q[t, hq])
                w = 2.0 ** (s - float(lse2[t, hq]))
                out[b, hq // G, pos[keep]] += w
                e = math.log(2) * (D * 2.0 ** -23 * scale * LOG2E * (np.abs(k) @ np.abs(q[t, hq])) + 2.0 ** -22 * (np.abs(s) + abs(float(lse2[t, hq])))) + 2.0 ** -21
                err[b, hq // G, pos[keep]] += w * e
    return out, bad, err


def evict_keep(w, L, budget, sinks, recent):
    """Positions that one KV head keeps, ascending.  w: its weights, float32."""
    if L <= budget:
        return list(range(L))
    mid = sorted(range(sinks, L - recent), key=lambda j: (-math.inf if math.isnan(w[j]) else float(w[j]), -j), reverse=True)
    # NaN is below -inf: sort those behind
    mid = [j for j in mid if not math.isnan(w[j])] + sorted(j for j in mid if math.isnan(w[j]))
    return sorted(list(range(sinks)) + mid[:budget - sinks - recent] + list(range(L - recent, L)))


def evict_tokens(Hkv, P, D, pools, page_codec, block_table, seq_lens, weights, budget, sinks, recent, codec, dst_codes, dst_meta, dst_table, row_len_out):
    """dst_codes / dst_meta (alloc_pool's layout) are updated in place.  Returns lengths, kept, weights_out, anomalies."""
    B = len(seq_lens)
    cap = block_table.shape[1] * P
    kept = np.full((B, Hkv, budget), -1, np.int32)
    w_out = np.zeros((B, Hkv, row_len_out), np.float32)
    lens, bad = [], 0
    for b in range(B):
        L = max(0, min(int(seq_lens[b]), cap))
        m = min(L, budget)
        lens.append(m)
        n_pages = (m + P - 1) // P
        x = np.zeros((2, Hkv, n_pages * P, D))
        raw = np.zeros((2, Hkv, n_pages * P, D), np.uint16)
        same = np.zeros((Hkv, n_pages * P), bool)
        for h in range(Hkv):
            ks = evict_keep(weights[b, h], L, budget, sinks, recent)
            kept[b, h, :m] = ks
            w_out[b, h, :m] = weights[b, h, ks]
            for i, j in enumerate(ks):
                c, slot = int(page_codec[b, j // P]), int(block_table[b, j // P])
                if c not in pools or not 0 <= slot < pools[c][0].shape[0]:
                    bad += 1
                    continue
                codes, meta = pools[c]
                for kv in range(2):
                    x[kv, h, i] = dequant_page(c, codes[slot:slot + 1], None if meta is None else meta[slot:slot + 1], 0, kv, h)[j % P]
                    if c == codec and c <= CODEC_BF16:
                        raw[kv, h, i] = codes[slot, kv, h, j % P]
                if c == codec and c <= CODEC_BF16:
                    same[h, i] = True
        for p in range(n_pages):
            slot = int(dst_table[b, p])
            if not 0 <= slot < dst_codes.shape[0]:
                bad += 1
                continue
            for kv in range(2):
                for h in range(Hkv):
                    y = x[kv, h, p * P:(p + 1) * P].astype(np.float32)
                    if codec == CODEC_FP16:
                        y = y.astype(np.float16).view(np.uint16)
                    elif codec == CODEC_BF16:
                        y = f64_to_bf16_bits(y.astype(np.float64))
                    elif codec == CODEC_FP8_E4M3:
                        y, dst_meta[slot, kv, h] = quantize_unit_fp8(y)
                    else:
                        assert codec == CODEC_INT8
                        y, dst_meta[slot, kv, h] = quantize_unit_int8(y)
                        y = y.view(np.uint8)
                    if codec <= CODEC_BF16:
                        y = np.where(same[h, p * P:(p + 1) * P, None], raw[kv, h, p * P:(p + 1) * P], y)
                    dst_codes[slot, kv, h] = y
    return np.array(lens), kept, w_out, bad
