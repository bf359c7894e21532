"""Differential attention without a GPU: exports, refusals, and the oracle
against independent forms of the same mathematics."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from oracle import diff_oracle as D
from paged_latent_attention_cache_gb300 import build, workloads as W

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def B():
    build.build()
    from paged_latent_attention_cache_gb300 import binding
    return binding


def _params(B, **kw):
    base = dict(dtype=B.PA_DTYPE_BF16, num_heads=8, kv_num_heads=2, head_size=64, rotary_dim=64,
                cos_rows=256, block_size=16, num_blocks=8, max_blocks_per_seq=4, lambda_init=0.3)
    base.update(kw)
    return B.make_diff_params(**base)


def test_exports_match_header(B):
    src = open(os.path.join(ROOT, "include", "pa_diff.h")).read()
    declared = sorted(set(re.findall(r"\b(pa_diff_\w+)\s*\(", src)))
    assert declared == sorted(B.EXPORTED_DIFF)
    for name in declared:
        assert hasattr(B.lib, name)


@pytest.mark.parametrize("kw", [
    {}, dict(v_head_size=0), dict(v_head_size=256), dict(head_size=128), dict(head_size=16, rotary_dim=0),
    dict(v_head_size=8), dict(scale=0.2), dict(num_heads=256, kv_num_heads=2), dict(softcap=30.0),
    dict(lambda_init=-0.5)])
def test_params_accepted(B, kw):
    assert B.pa_diff_validate(_params(B, **kw)) == B.PA_OK, B.last_error()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=7), 2, "float16"), (dict(num_heads=0), 1, "num_heads"),
    (dict(kv_num_heads=3), 1, "kv_num_heads"), (dict(kv_num_heads=0), 1, "kv_num_heads"),
    (dict(head_size=72), 1, "multiple of 16"), (dict(head_size=144), 2, "head_size"),
    (dict(v_head_size=-8), 1, "v_head_size"), (dict(v_head_size=260), 2, "v_head_size"),
    (dict(v_head_size=264), 2, "v_head_size"), (dict(v_head_size=12), 2, "v_head_size"),
    (dict(num_heads=258, kv_num_heads=2), 2, "heads"),
    (dict(rotary_dim=80), 1, "exceeds"), (dict(rotary_dim=8), 1, "multiple of 16"),
    (dict(cos_rows=0), 1, "cos_rows"), (dict(block_size=24), 1, "power of two"),
    (dict(scale=-1.0), 1, "scale"), (dict(scale=float("nan")), 1, "scale"),
    (dict(softcap=float("inf")), 1, "softcap"), (dict(lambda_init=float("nan")), 1, "lambda_init"),
    (dict(lambda_init=float("inf")), 1, "lambda_init"), (dict(norm_eps=-1e-5), 1, "norm_eps"),
    (dict(norm_eps=float("nan")), 1, "norm_eps"), (dict(flags=1), 1, "flag"), (dict(flags=8), 1, "flag"),
    (dict(num_heads=65536, kv_num_heads=65536), 2, "65535"),
    (dict(num_blocks=0), 1, "num_blocks"), (dict(max_blocks_per_seq=0), 1, "max_blocks_per_seq"),
])
def test_params_refused(B, kw, status, needle):
    p = _params(B, **kw)
    assert B.pa_diff_validate(p) == status
    assert needle in B.last_error()
    assert B.pa_diff_workspace_size(p, 4, 4) == 0


def _read(Bm, fn, **over):
    a = dict(q=0x10000, T=8, kc=0x20000, vc=0x28000, cos=0x30000, sin=0x40000, lv=0x44000, nw=0x48000,
             cumseq=0x50000, past=0x60000, bt=0x70000, B=2, sb=0, se=2, ws=0x100000, wsb=1 << 40, out=0x80000,
             err=0x90000)
    a.update(over)
    vp = lambda x: ctypes.c_void_p(x) if x else None
    return fn(ctypes.byref(_params(Bm)), vp(a["q"]), a["T"], vp(a["kc"]), vp(a["vc"]), vp(a["cos"]), vp(a["sin"]),
              vp(a["lv"]), vp(a["nw"]), vp(a["cumseq"]), vp(a["past"]), vp(a["bt"]), a["B"], a["sb"], a["se"],
              vp(a["ws"]), ctypes.c_size_t(a["wsb"]), vp(a["out"]), vp(a["err"]), None)


@pytest.mark.parametrize("over,needle", [
    (dict(q=0), "NULL"), (dict(kc=0), "NULL"), (dict(vc=0), "NULL"), (dict(lv=0), "NULL"), (dict(nw=0), "NULL"),
    (dict(bt=0), "NULL"), (dict(out=0), "NULL"), (dict(cos=0), "cos_cache"), (dict(q=0x10008), "16-byte"),
    (dict(vc=0x28008), "16-byte"), (dict(nw=0x48002), "16-byte"), (dict(lv=0x44002), "4-byte"),
    (dict(cumseq=0x50002), "4-byte"), (dict(sb=1, se=3), "sequence range"), (dict(sb=-1), "sequence range"),
    (dict(T=-1), "num_tokens"), (dict(T=1 << 30), "num_tokens"), (dict(B=-1), "num_"), (dict(ws=0x100010), "256-byte"),
])
def test_read_refused(B, over, needle):
    for fn in (B.lib.pa_diff_decode, B.lib.pa_diff_prefill):
        assert _read(B, fn, **over) == B.PA_ERR_INVALID_ARGUMENT, (over, B.last_error())
        assert needle in B.last_error()


def test_read_nothing_to_do(B):
    for fn in (B.lib.pa_diff_decode, B.lib.pa_diff_prefill):
        assert _read(B, fn, T=0) == B.PA_OK
        assert _read(B, fn, sb=1, se=1) == B.PA_OK
    assert _read(B, B.lib.pa_diff_decode, T=1) == B.PA_ERR_INVALID_ARGUMENT


def test_write_refused(B):
    vp = ctypes.c_void_p
    good = [vp(0x10000), vp(0x18000), 4, vp(0x20000), vp(0x30000), vp(0x40000), vp(0x50000), vp(0x60000), 2,
            vp(0x70000), vp(0x80000), vp(0x90000), None]
    p = _params(B)
    for i, v, needle in [(0, None, "NULL"), (1, None, "NULL"), (9, None, "NULL"), (3, None, "cos_cache"),
                         (1, vp(0x18008), "16-byte"), (10, vp(0x80004), "16-byte"), (5, vp(0x40002), "4-byte"),
                         (8, 0, "num_seqs"), (2, -1, "num_tokens")]:
        a = list(good)
        a[i] = v
        assert B.lib.pa_diff_write(ctypes.byref(p), *a) == B.PA_ERR_INVALID_ARGUMENT
        assert needle in B.last_error(), (i, B.last_error())
    good[2] = 0
    assert B.lib.pa_diff_write(ctypes.byref(p), *good) == B.PA_OK


# ---- the oracle

def _numpy(w):
    t = {}
    for k, v in w.tensors.items():
        t[k] = W.to_bits(v) if v.dtype in (torch.bfloat16, torch.float16) else v.numpy()
    return t


def test_oracle_equals_dense_torch():
    """Contiguous dense differential attention in torch float64, no paging."""
    w = W.make_diff_workload("d", [5, 9], [0, 0], num_heads=4, kv_num_heads=2, head_size=32, block_size=16,
                             rotary_dim=0, seed=3, lambda_init=0.4)
    ref = D.run_bits(_numpy(w), w.params, "bf16")
    d = lambda k: w.tensors[k].double()
    lv = d("lambda_vectors")
    la = torch.exp(lv[0] @ lv[1]) - torch.exp(lv[2] @ lv[3]) + 0.4
    at = 0
    for q in (5, 9):
        Q = d("query")[at:at + q].view(q, 4, 2, 32)
        K = d("key")[at:at + q].view(q, 2, 2, 32).repeat_interleave(2, 1)
        V = d("value")[at:at + q].view(q, 2, 64).repeat_interleave(2, 1)
        s = torch.einsum("qhid,khid->hiqk", Q, K) / 32 ** 0.5
        s = s.masked_fill(torch.ones(q, q).triu(1).bool(), float("-inf")).softmax(-1)
        o = torch.einsum("hqk,khd->qhd", s[:, 0] - la * s[:, 1], V)
        o = torch.nn.functional.rms_norm(o, (64,), d("norm_weight"), 1e-5) * 0.6
        assert np.allclose(ref["out"][at:at + q], o.numpy(), rtol=1e-9, atol=1e-11)
        at += q


def test_oracle_closed_forms():
    """One key: both maps are 1, so o = (1 - lambda) V. Equal keys in both maps
    and lambda = 1: the maps cancel and the output is 0."""
    w = W.make_diff_workload("d", [1], [0], num_heads=2, kv_num_heads=1, head_size=16, block_size=16, seed=1)
    t = _numpy(w)
    ref = D.run_bits(t, w.params, "bf16")
    v = w.tensors["value"].double().numpy().reshape(32)
    sign = np.sign(1 - D.lam(t["lambda_vectors"], 0.5))
    want = 0.5 * w.tensors["norm_weight"].double().numpy() * sign * v / np.sqrt((v * v).mean())
    assert np.allclose(ref["out"][0], want, rtol=1e-3)  # norm_eps beside ((1 - lambda) v)^2
    w = W.make_diff_workload("d", [3], [0], num_heads=1, kv_num_heads=1, head_size=16, block_size=16, seed=1,
                             lambda_init=1.0, rotary_dim=0)
    for k in ("query", "key"):
        x = w.tensors[k].view(3, 2, 16)
        x[:, 1] = x[:, 0]
    w.tensors["lambda_vectors"].zero_()
    assert np.abs(D.run_bits(_numpy(w), w.params, "bf16")["out"]).max() < 1e-12


def test_oracle_noise_is_the_spread_of_rounded_runs():
    """Rounding the probabilities and queries of a dense run at random moves
    the outputs by about the predicted amount (within a factor of two over
    all outputs, never more than six times it for one)."""
    w = W.make_diff_workload("d", [1], [60], num_heads=2, kv_num_heads=1, head_size=32, block_size=16,
                             rotary_dim=0, seed=5, lambda_init=0.6)
    t = _numpy(w)
    ref = D.run_bits(t, w.params, "bf16")
    d = lambda k: w.tensors[k].double().numpy()
    rows = (w.tensors["block_table"].numpy()[0, np.arange(61) // 16] * 16 + np.arange(61) % 16)
    kc = d("key_cache").reshape(-1, 2, 32)
    vc = d("value_cache").reshape(-1, 64)
    kc[rows[60]], vc[rows[60]] = d("key").reshape(2, 32), d("value").reshape(64)
    K, V, Q = kc[rows], vc[rows], d("query").reshape(2, 2, 32)
    rng, u = np.random.default_rng(0), 2.0 ** -8
    err = []
    for _ in range(200):
        o = []
        for i in range(2):
            q = Q[:, i] * (1 + u * rng.uniform(-1, 1, size=Q[:, i].shape))
            p = np.exp(q @ K[:, i].T / 32 ** 0.5)
            o.append((p * (1 + u * rng.uniform(-1, 1, size=p.shape))) @ V / p.sum(-1, keepdims=True))
        got = D.combine(o[0], o[1], t["lambda_vectors"], d("norm_weight"), 0.6, 1e-5)
        err.append(got - ref["out"][0])
    err = np.array(err)
    predicted = u * (ref["noise"][0] - np.abs(ref["out"][0]))
    spread = np.sqrt(3) * err.std(0)
    assert (np.abs(err) < 6 * u * ref["noise"][0]).all()
    assert 0.5 < np.sqrt((spread ** 2).sum() / (predicted ** 2).sum()) < 2.0
