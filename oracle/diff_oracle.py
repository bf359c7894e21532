"""CPU oracle for differential attention (include/pa_diff.h).

TEST INFRASTRUCTURE ONLY, float64. Each of the two softmax maps is the
SEPARATE-layout attention of ``pa_oracle`` (pinned there) over that map's
keys; this file adds what is new: the difference with lambda, the norm and
the bound on a kernel's rounding errors."""
from __future__ import annotations

import math

import numpy as np

from oracle import pa_oracle as P


def lam(vectors: np.ndarray, lambda_init: float) -> float:
    v = np.asarray(vectors, dtype=np.float64)
    return math.exp(float(v[0] @ v[1])) - math.exp(float(v[2] @ v[3])) + lambda_init


def combine(o0, o1, vectors, norm_weight, lambda_init, eps):
    """(1 - lambda_init) * w * o / rms(o), o = o0 - lambda * o1, over the last axis."""
    o = o0 - lam(vectors, lambda_init) * o1
    r = np.sqrt((o * o).mean(-1, keepdims=True) + eps)
    return (1.0 - lambda_init) * norm_weight * o / r


def run_bits(t: dict, p: dict, dtype: str, tokens=None):
    """``t``: the tensors as numpy arrays (half-precision ones as uint16
    bits), ``p``: the operator's parameters. Write then read. Returns a dict
    with the cache bits, ``out`` [tokens, H, vhs] in float64 and ``noise``:
    per output, how far independent roundings of the probabilities and of the
    query operand (relative size 1) move it, in standard deviations times
    sqrt(3), plus the rounding of the output itself."""
    H, kv, hs = p["num_heads"], p["kv_num_heads"], p["head_size"]
    vhs = p["v_head_size"] or 2 * hs
    f = lambda k: P.bits_to_f64(t[k], dtype)
    q = dict(p, num_heads=H, kv_num_heads=kv, v_head_size=vhs, scale=p["scale"] or hs ** -0.5,
             rms_eps=0.0)
    cos, sin = f("cos_cache"), f("sin_cache")
    kc = [P.BitsCache(t["key_cache"][:, :, :, i].reshape(-1, hs), dtype) for i in range(2)]
    vc = P.BitsCache(t["value_cache"].reshape(-1, vhs), dtype)
    key, value = f("key").reshape(-1, kv, 2, hs), f("value").reshape(-1, kv, vhs)
    for i in range(2):
        P.separate_write(lambda n, i=i: key[n][:, i], lambda n: value[n], cos, sin,
                         t["slot_mapping"], t["cumseq"], t["past"], kc[i], vc, q)
    tokens = range(int(t["cumseq"][-1])) if tokens is None else tokens
    query = f("query").reshape(-1, H, 2, hs)
    w, lv = f("norm_weight"), t["lambda_vectors"]
    la = lam(lv, p["lambda_init"])
    outs, noise = [], []
    for n in tokens:
        o, s = [], []
        for i in range(2):
            oi, si = P.separate_attend_token(int(n), query[n][:, i].reshape(-1), kc[i], vc, cos,
                                             sin, t["cumseq"], t["past"], t["block_table"], q,
                                             stats=True)
            o.append(oi)
            s.append(np.sqrt(si[0] ** 2 + si[1] ** 2))
        d = o[0] - la * o[1]
        e = np.sqrt(s[0] ** 2 + (la * s[1]) ** 2)  # of the difference
        out = combine(o[0], o[1], lv, w, p["lambda_init"], p["norm_eps"])
        r = np.sqrt((d * d).mean(-1, keepdims=True) + p["norm_eps"])
        # the norm divides by r, whose own relative error is that of an average
        # over the channels of d * e / r^2
        rel = np.sqrt(((d * e) ** 2).sum(-1, keepdims=True)) / (vhs * r * r)
        gain = np.abs((1.0 - p["lambda_init"]) * w) / r
        outs.append(out)
        noise.append(np.sqrt((gain * e) ** 2 + (np.abs(out) * rel) ** 2) + np.abs(out))
    kcb = np.stack([c.bits.reshape(t["key_cache"].shape[:3] + (hs,)) for c in kc], axis=3)
    return dict(key_cache=kcb, value_cache=vc.bits.reshape(t["value_cache"].shape),
                out=np.stack(outs), noise=np.stack(noise))
