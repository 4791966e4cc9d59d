"""CPU oracle of the 8-bit latent cache and of key selection, in float64.

Written from the definitions in include/mla_prefill.h: a cache of e4m3 codes
with a power-of-two scale for each block of slots, absorbed decode over its
values, key scores and block selection.  Plain loops; no kernel's order.
"""
from __future__ import annotations

import math

import numpy as np

from .mla_oracle import DN, R, e4m3_decode, e4m3_encode, rms_norm, rope_rotate

SCALE_MIN_EXP, SCALE_MAX_EXP = -60, 120


def block_scale(amax: float) -> float:
    """The smallest power of two s with amax <= 448 s, between 2**-60 and 2**120."""
    if not amax > 0:
        return 2.0 ** SCALE_MIN_EXP
    if math.isinf(amax):
        return 2.0 ** SCALE_MAX_EXP
    e = math.frexp(amax / 448.0)
    exp = e[1] - 1 if e[0] == 0.5 else e[1]
    return 2.0 ** max(SCALE_MIN_EXP, min(SCALE_MAX_EXP, exp))


def q8_values(codes, scales, scale_block: int):
    """Real values [rows, 576] of a cache [num_pages, page_size, 576]."""
    rows = np.asarray(codes).reshape(-1, codes.shape[-1])
    return e4m3_decode(rows) * np.repeat(np.asarray(scales, np.float64).reshape(-1), scale_block)[:, None]


def new_rows(kv_latent, kv_norm_gamma, freqs_cis, input_row_offsets, cache_lengths, epsilon):
    """Values before quantisation of every new token's row, [T, 576]."""
    lat = np.asarray(kv_latent, np.float64)
    y = np.full(lat.shape, np.nan)
    iro = np.asarray(input_row_offsets, np.int64)
    for b, p in enumerate(np.asarray(cache_lengths, np.int64)):
        for t in range(iro[b], iro[b + 1]):
            y[t, :R] = rms_norm(lat[t, :R], kv_norm_gamma, epsilon)
            y[t, R:] = rope_rotate(lat[t, R:], freqs_cis[p + t - iro[b]])
    return y


def latent_cache_write_q8(kv_codes, kv_scales, y, input_row_offsets, cache_lengths, page_table, page_size: int,
                          scale_block: int):
    """Quantise the rows ``y`` (new_rows) into the cache block by block.
    Returns (codes, scales, unrounded codes y / s of the rows written [T, 576])."""
    codes, scales = np.array(kv_codes, copy=True), np.array(kv_scales, np.float64, copy=True).reshape(-1)
    flat = codes.reshape(-1, codes.shape[-1])
    iro = np.asarray(input_row_offsets, np.int64)
    pre = np.full(y.shape, np.nan)
    for b, p in enumerate(np.asarray(cache_lengths, np.int64)):
        n = int(iro[b + 1] - iro[b])
        i = 0
        while i < n:
            pos = int(p) + i
            slot = pos % scale_block
            m = min(scale_block - slot, n - i)
            row = int(page_table[b][pos // page_size]) * page_size + pos % page_size
            rows = y[iro[b] + i: iro[b] + i + m]
            s = block_scale(float(np.nanmax(np.abs(rows), initial=0.0)))
            was = scales[row // scale_block]
            if slot > 0 and was > 0 and math.isfinite(was):
                if was >= s:
                    s = was
                else:
                    flat[row - slot: row] = e4m3_encode(e4m3_decode(flat[row - slot: row]) * (was / s))
            scales[row // scale_block] = s
            pre[iro[b] + i: iro[b] + i + m] = rows / s
            flat[row: row + m] = e4m3_encode(rows / s)
            i += m
    return codes, scales.reshape(np.shape(kv_scales)), pre


def absorbed_attention(u, rows, w_uv, scale: float, sink=None, visible=None):
    """One token: u [H, 576] absorbed queries, rows [n, 576] values, w_uv
    [H, 128, 512]; visible bool [n].  Returns (out [H, 128], lse [H])."""
    rows = np.asarray(rows, np.float64)
    if visible is not None:
        rows = rows[visible]
    s = scale * (np.asarray(u, np.float64) @ rows.T)
    if sink is not None:
        s = np.concatenate([s, np.full((s.shape[0], 1), float(sink))], 1)
    if s.shape[1] == 0:
        return np.zeros((s.shape[0], w_uv.shape[1])), np.full(s.shape[0], -np.inf)
    top = s.max(1, keepdims=True)
    e = np.exp(s - top)
    tot = e.sum(1, keepdims=True)
    o = (e / tot)[:, : rows.shape[0]] @ rows[:, :R]
    return np.einsum("hk,hdk->hd", o, w_uv), top[:, 0] + np.log(tot[:, 0])


def decode_values(q, values, page_table, page_size: int, w_uk, w_uv, input_row_offsets, cache_lengths, scale,
                  indices=None, topk_lengths=None, attn_sink=None):
    """mla_decode_q8 on real cache values [rows, 576]: out [T, H, 128], lse [T, H]
    (NaN for tokens outside every sequence)."""
    q = np.asarray(q, np.float64)
    T, H = q.shape[:2]
    out, lse = np.full((T, H, w_uv.shape[1]), np.nan), np.full((T, H), np.nan)
    iro = np.asarray(input_row_offsets, np.int64)
    for b in range(len(iro) - 1):
        n, p = int(iro[b + 1] - iro[b]), int(cache_lengths[b])
        if n <= 0:
            continue
        if indices is None:
            j = np.arange(p + n)
            row = np.asarray(page_table[b], np.int64)[j // page_size] * page_size + j % page_size
        else:
            k = indices.shape[1] if topk_lengths is None else max(0, min(int(topk_lengths[b]), indices.shape[1]))
            row = np.asarray(indices[b][:k], np.int64)
        ctx = values[row]
        for i in range(n):
            t = int(iro[b]) + i
            u = np.concatenate([np.einsum("hd,hkd->hk", q[t, :, :DN], w_uk), q[t, :, DN:]], 1)
            rows = ctx if indices is not None else ctx[: p + i + 1]
            out[t], lse[t] = absorbed_attention(u, rows, w_uv, scale, None if attn_sink is None else attn_sink[b])
    return out, lse


def index_scores(index_q, index_w, index_keys, index_scales, page_table, page_size: int, input_row_offsets,
                 cache_lengths, block: int, stride: int):
    """Block scores [T, stride] (NaN rows outside every sequence), and for the
    rounding bound the sum over h of |w| times sum |q||k|, maximised over the
    block like the score."""
    q, w = np.asarray(index_q, np.float64), np.asarray(index_w, np.float64)
    keys = np.asarray(index_keys, np.float64).reshape(-1, q.shape[-1])
    T = q.shape[0]
    got, mag = np.full((T, stride), np.nan), np.zeros((T, stride))
    iro = np.asarray(input_row_offsets, np.int64)
    for b in range(len(iro) - 1):
        for t in range(int(iro[b]), int(iro[b + 1])):
            P = int(cache_lengths[b]) + t - int(iro[b])
            j = np.arange(P + 1)
            row = np.asarray(page_table[b], np.int64)[j // page_size] * page_size + j % page_size
            ks = 1.0 if index_scales is None else np.asarray(index_scales, np.float64)[row]
            x = (np.maximum(q[t] @ keys[row].T, 0) * w[t][:, None]).sum(0) * ks
            m = ((np.abs(q[t]) @ np.abs(keys[row]).T) * np.abs(w[t])[:, None]).sum(0) * ks
            pad = -(P + 1) % block
            x = np.concatenate([x, np.full(pad, -np.inf)]).reshape(-1, block).max(1)
            m = np.concatenate([m, np.zeros(pad)]).reshape(-1, block).max(1)
            got[t] = -np.inf
            got[t, : len(x)], mag[t, : len(m)] = x, m
    return got, mag


def index_select(scores, page_table, page_size: int, input_row_offsets, cache_lengths, block: int, top: int,
                 local: int, stride: int):
    """(indices [T, stride] int, counts [T]); rows of tokens outside every
    sequence are None in the list of lists."""
    scores = np.asarray(scores, np.float64)
    T = scores.shape[0]
    lists, counts = [None] * T, [None] * T
    iro = np.asarray(input_row_offsets, np.int64)
    for b in range(len(iro) - 1):
        for t in range(int(iro[b]), int(iro[b + 1])):
            P = int(cache_lengths[b]) + t - int(iro[b])
            nb = P // block + 1
            s = np.where(np.isnan(scores[t, :nb]), -np.inf, scores[t, :nb])
            always = [x for x in range(nb) if x >= nb - local]
            rest = sorted((x for x in range(nb) if x < nb - local), key=lambda x: (-s[x], x))
            chosen = sorted((always + rest)[: min(top, nb)]) if local else sorted(rest[: min(top, nb)])
            pos = [j for x in chosen for j in range(x * block, min((x + 1) * block, P + 1))]
            row = [int(page_table[b][j // page_size]) * page_size + j % page_size for j in pos]
            lists[t] = row + [-1] * (stride - len(row))
            counts[t] = len(row)
    return lists, counts
