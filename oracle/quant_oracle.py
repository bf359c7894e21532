"""CPU oracle for paged caches in 8 bits (include/pa_quant.h).

TEST INFRASTRUCTURE ONLY, float64, token by token. E4M3, the rotation and the
norm are those of ``pa_oracle`` (pinned there); this file adds the scales, their
growth, reading back, cross attention and the bound on a kernel's roundings."""
from __future__ import annotations

import math

import numpy as np

from oracle import pa_oracle as P

LEAST, MOST = -48, 48


def exponent_for(amax: float) -> int:
    """The least e in [LEAST, MOST] with amax <= 448 * 2^e (MOST where none is enough)."""
    e = LEAST
    while e < MOST and amax > math.ldexp(448.0, e):
        e += 1
    return e


def stored(scale: float) -> float:
    """A scale as it counts: a power of two in range, or 0."""
    scale = float(scale)
    if not (math.isfinite(scale) and scale > 0):
        return 0.0
    m, e = math.frexp(scale)
    return scale if m == 0.5 and LEAST <= e - 1 <= MOST else 0.0


def encode(x: np.ndarray) -> np.ndarray:
    """E4M3 codes; NaN becomes 0x7f, infinities saturate."""
    x = np.asarray(x, dtype=np.float64)
    return np.where(np.isnan(x), np.uint8(0x7F), P.round_to_e4m3(np.nan_to_num(x, nan=0.0)))


def write(key, value, cos, sin, slots, cumseq, past, kc, vc, scales, p, k_norm=None):
    """``key`` [T, kv, hs], ``value`` [T, kv, vhs] float64; ``kc``, ``vc`` uint8 [blocks, bs, kv, .] and
    ``scales`` float32 [blocks, kv, 2], updated in place. Keys are rounded to float32 before they are
    encoded."""
    bs, blocks = p["block_size"], kc.shape[0]
    for b in range(len(past)):
        pages = {}  # logical page -> [page, {row: token}]
        for t in range(int(cumseq[b]), int(cumseq[b + 1])):
            pos, slot = int(past[b]) + t - int(cumseq[b]), int(slots[t])
            if pos < 0 or slot < 0 or slot >= blocks * bs or slot % bs != pos % bs:
                continue
            if p["rotary_dim"] and pos >= p["cos_rows"]:
                continue
            page, rows = pages.setdefault(pos // bs, (slot // bs, {}))
            if slot // bs == page:
                rows[slot % bs] = (t, pos)
        for page, rows in pages.values():
            for g in range(p["kv_num_heads"]):
                new = [{}, {}]
                for r, (t, pos) in rows.items():
                    k = key[t, g] if k_norm is None else P.rms_norm(key[t, g], k_norm, p["rms_eps"])
                    k = P.rope_row(k, pos, p["rotary_offset"], p["rotary_dim"], cos, sin,
                                   bool(p["rotary_interleaved"]))
                    new[0][r], new[1][r] = k.astype(np.float32).astype(np.float64), value[t, g]
                for i, cache in enumerate((kc, vc)):
                    amax = max(np.abs(x[np.isfinite(x)]).max(initial=0.0) for x in new[i].values())
                    old = 0.0 if 0 in rows else stored(scales[page, g, i])
                    scale = max(old, math.ldexp(1.0, exponent_for(amax)))
                    if 0 < old < scale:
                        cache[page, :, g] = encode(P.e4m3_to_f64(cache[page, :, g]) * (old / scale))
                    scales[page, g, i] = scale
                    for r, x in new[i].items():
                        cache[page, r, g] = encode(x / scale)


def rows_of(cache, scales, i, pages, rows, g):
    s = np.array([stored(x) for x in scales[pages, g, i]])
    with np.errstate(invalid="ignore"):
        return P.e4m3_to_f64(cache[pages, rows, g]) * s[:, None]


def attend(query, kc, vc, scales, cos, sin, cumseq, past, table, p, head_sink=None, q_norm=None):
    """``query`` [T, H, hs] float64. Returns out [T, H, vhs] and the bound on a kernel's error, from its
    roundings: the output's own (at most u |out|, u = 2^-8 or 2^-11); those of the fp16 operands, taken
    as independent, six times their root sum of squares with 2^-11 each (probabilities n_p, query n_q);
    f32 accumulation, which may cut off 2^-23 in each of n / 16 additions of 16 keys; and the fp16 floor
    of probabilities, 2^-36 of the row's largest product of probability and scale for each key (an eighth
    of what the header allows: half of fp16's least step 2^-24 against a largest product of 2^8 or more)."""
    H, kv, hs = p["num_heads"], p["kv_num_heads"], p["head_size"]
    vhs, bs = p["v_head_size"] or hs, p["block_size"]
    scale = p["scale"] or hs ** -0.5
    u = 2.0 ** (-8 if p["dtype"] == P.BF16 else -11)
    T = query.shape[0]
    out, tol = np.zeros((T, H, vhs)), np.zeros((T, H, vhs))
    for t in range(int(cumseq[-1])):
        b, pos = P.locate_token(t, cumseq, past)
        last = int(past[b]) - 1 if p["cross"] else pos
        lo = max(0, last - p["local_window_size"]) if p["local_window_size"] >= 0 else 0
        j = np.arange(lo, last + 1)
        if not len(j):
            continue
        pages, rows = table[b, j // bs], j % bs
        for g in range(kv):
            K, V = rows_of(kc, scales, 0, pages, rows, g), rows_of(vc, scales, 1, pages, rows, g)
            vs = np.array([stored(x) for x in scales[pages, g, 1]])
            codes = np.abs(P.e4m3_to_f64(vc[pages, rows, g]))
            for h in range(g * (H // kv), (g + 1) * (H // kv)):
                q = query[t, h] if q_norm is None else P.rms_norm(query[t, h], q_norm, p["rms_eps"])
                q = P.rope_row(q, pos, p["rotary_offset"], p["rotary_dim"], cos, sin,
                               bool(p["rotary_interleaved"])) if p["rotary_dim"] else q
                s = K @ q * scale
                if p["softcap"] > 0:
                    s = p["softcap"] * np.tanh(s / p["softcap"])
                m = s.max()
                w = np.exp(s - m)
                den = w.sum() + (0.0 if head_sink is None else np.exp(head_sink[h] - m))
                prob = w / den
                o = prob @ V
                out[t, h] = o
                n = P.error_scales_kv(q[None], K, V, prob[None], o[None], scale)[:, 0]
                tol[t, h] = (u * np.abs(o) + 6 * 2.0 ** -11 * np.sqrt(n[0] ** 2 + n[1] ** 2)
                             + (len(j) / 16 + 1) * 2.0 ** -23 * (prob @ np.abs(V))
                             + 2.0 ** -36 * (prob * vs).max() * codes.sum(0))
    return out, tol
