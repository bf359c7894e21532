"""Paged caches in 8 bits without a GPU: exports, refusals, and the oracle against independent forms
of the same mathematics."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from oracle import pa_oracle as P, quant_oracle as Q
from paged_latent_attention_cache_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def B():
    build.build()
    from paged_latent_attention_cache_gb300 import binding
    return binding


def _params(B, **kw):
    base = dict(dtype=B.PA_DTYPE_BF16, num_heads=8, kv_num_heads=2, head_size=64, rotary_dim=64,
                cos_rows=256, block_size=16, num_blocks=8, max_blocks_per_seq=4)
    base.update(kw)
    return B.make_quant_params(**base)


def test_exports_match_header(B):
    src = open(os.path.join(ROOT, "include", "pa_quant.h")).read()
    declared = sorted(set(re.findall(r"\b(pa_quant_\w+)\s*\(", src)))
    assert declared == sorted(B.EXPORTED_QUANT)
    for name in declared:
        assert hasattr(B.lib, name)


@pytest.mark.parametrize("kw", [
    {}, dict(v_head_size=0), dict(v_head_size=256), dict(head_size=256), dict(head_size=16, rotary_dim=0),
    dict(v_head_size=16), dict(scale=0.2), dict(num_heads=256, kv_num_heads=2), dict(softcap=30.0),
    dict(block_size=4096), dict(cross=1, rotary_dim=0), dict(local_window_size=0), dict(rotary_dim=32, rotary_offset=8)])
def test_params_accepted(B, kw):
    assert B.pa_quant_validate(_params(B, **kw)) == B.PA_OK, B.last_error()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=7), 2, "float16"), (dict(num_heads=0), 1, "num_heads"),
    (dict(kv_num_heads=3), 1, "kv_num_heads"), (dict(kv_num_heads=0), 1, "kv_num_heads"),
    (dict(head_size=72), 1, "multiple of 16"), (dict(head_size=272), 2, "head_size"),
    (dict(v_head_size=-16), 1, "v_head_size"), (dict(v_head_size=24), 2, "v_head_size"),
    (dict(v_head_size=272), 2, "v_head_size"), (dict(num_heads=258, kv_num_heads=2), 2, "heads"),
    (dict(rotary_dim=80), 1, "exceeds"), (dict(rotary_dim=8), 1, "multiple of 16"),
    (dict(rotary_dim=32, rotary_offset=4), 1, "multiple of 8"),
    (dict(cos_rows=0), 1, "cos_rows"), (dict(block_size=24), 1, "power of two"), (dict(block_size=8192), 2, "block_size"),
    (dict(scale=-1.0), 1, "scale"), (dict(scale=float("nan")), 1, "scale"),
    (dict(softcap=float("inf")), 1, "softcap"), (dict(rms_eps=-1.0), 1, "rms_eps"),
    (dict(cross=2), 1, "cross"), (dict(cross=1), 1, "cross"), (dict(cross=1, rotary_dim=0, local_window_size=4), 1, "cross"),
    (dict(flags=1), 1, "flag"), (dict(flags=8), 1, "flag"),
    (dict(num_heads=65536, kv_num_heads=65536), 2, "65535"),
    (dict(num_blocks=0), 1, "num_blocks"), (dict(max_blocks_per_seq=0), 1, "max_blocks_per_seq"),
])
def test_params_refused(B, kw, status, needle):
    p = _params(B, **kw)
    assert B.pa_quant_validate(p) == status
    assert needle in B.last_error()
    assert B.pa_quant_workspace_size(p, 4, 4) == 0


def _vp(x):
    return ctypes.c_void_p(x) if x else None


def _read(Bm, fn, **over):
    a = dict(q=0x10000, T=8, kc=0x20000, vc=0x28000, sc=0x2c000, cos=0x30000, sin=0x40000, qn=0, sink=0,
             cumseq=0x50000, past=0x60000, bt=0x70000, B=2, sb=0, se=2, ws=0x100000, wsb=1 << 40, out=0x80000,
             err=0x90000)
    a.update(over)
    return fn(ctypes.byref(_params(Bm)), _vp(a["q"]), a["T"], _vp(a["kc"]), _vp(a["vc"]), _vp(a["sc"]), _vp(a["cos"]),
              _vp(a["sin"]), _vp(a["qn"]), _vp(a["sink"]), _vp(a["cumseq"]), _vp(a["past"]), _vp(a["bt"]), a["B"],
              a["sb"], a["se"], _vp(a["ws"]), ctypes.c_size_t(a["wsb"]), _vp(a["out"]), _vp(a["err"]), None)


@pytest.mark.parametrize("over,needle", [
    (dict(q=0), "NULL"), (dict(kc=0), "NULL"), (dict(vc=0), "NULL"), (dict(sc=0), "NULL"), (dict(bt=0), "NULL"),
    (dict(out=0), "NULL"), (dict(cos=0), "cos_cache"), (dict(q=0x10008), "16-byte"), (dict(vc=0x28008), "16-byte"),
    (dict(sc=0x2c004), "8-byte"), (dict(qn=0x48002), "16-byte"), (dict(sink=0x48001), "16-byte"),
    (dict(cumseq=0x50002), "4-byte"), (dict(sb=1, se=3), "sequence range"), (dict(sb=-1), "sequence range"),
    (dict(T=-1), "num_tokens"), (dict(T=1 << 30), "num_tokens"), (dict(B=-1), "num_"), (dict(ws=0x100010), "256-byte"),
])
def test_read_refused(B, over, needle):
    for fn in (B.lib.pa_quant_decode, B.lib.pa_quant_prefill):
        assert _read(B, fn, **over) == B.PA_ERR_INVALID_ARGUMENT, (over, B.last_error())
        assert needle in B.last_error()


def test_read_nothing_to_do(B):
    for fn in (B.lib.pa_quant_decode, B.lib.pa_quant_prefill):
        assert _read(B, fn, T=0) == B.PA_OK
        assert _read(B, fn, sb=1, se=1) == B.PA_OK
    assert _read(B, B.lib.pa_quant_decode, T=1) == B.PA_ERR_INVALID_ARGUMENT


def test_write_and_restore_refused(B):
    vp = ctypes.c_void_p
    p = _params(B)
    good = [vp(0x10000), vp(0x18000), 4, vp(0x20000), vp(0x30000), None, vp(0x40000), vp(0x50000), vp(0x60000), 2,
            vp(0x70000), vp(0x80000), vp(0x88000), vp(0x90000), None]
    for i, v, needle in [(0, None, "NULL"), (1, None, "NULL"), (10, None, "NULL"), (12, None, "NULL"), (3, None, "cos_cache"),
                         (1, vp(0x18008), "16-byte"), (5, vp(0x18008), "16-byte"), (11, vp(0x80004), "16-byte"),
                         (12, vp(0x88004), "8-byte"), (6, vp(0x40002), "4-byte"), (9, 0, "num_seqs"), (2, -1, "num_tokens")]:
        a = list(good)
        a[i] = v
        assert B.lib.pa_quant_write(ctypes.byref(p), *a) == B.PA_ERR_INVALID_ARGUMENT
        assert needle in B.last_error(), (i, B.last_error())
    good[2] = 0
    assert B.lib.pa_quant_write(ctypes.byref(p), *good) == B.PA_OK
    good = [vp(0x10000), vp(0x18000), vp(0x20000), vp(0x30000), vp(0x40000), vp(0x50000), 2, 4, vp(0x70000), vp(0x80000),
            vp(0x90000), None]
    for i, v, needle in [(0, None, "NULL"), (2, None, "NULL"), (5, None, "NULL"), (8, vp(0x70008), "16-byte"),
                         (1, vp(0x18008), "16-byte"), (2, vp(0x20004), "8-byte"), (3, vp(0x30002), "4-byte"),
                         (6, 0, "num_seqs"), (7, -1, "num_tokens")]:
        a = list(good)
        a[i] = v
        assert B.lib.pa_quant_restore(ctypes.byref(p), *a) == B.PA_ERR_INVALID_ARGUMENT
        assert needle in B.last_error(), (i, B.last_error())
    good[8] = good[9] = None
    assert B.lib.pa_quant_restore(ctypes.byref(p), *good) == B.PA_OK  # nothing asked for


def test_mixed_refused(B):
    vp = ctypes.c_void_p
    good = [vp(0x10000), vp(0x18000), vp(0x20000), 4, vp(0x28000), vp(0x30000), None, None, None, vp(0x38000), vp(0x40000),
            vp(0x50000), vp(0x60000), 2, 1, vp(0x70000), vp(0x80000), vp(0x88000), vp(0x100000), ctypes.c_size_t(1 << 40),
            vp(0x90000), vp(0xa0000), None]
    for i, v, needle in [(0, None, "NULL"), (1, None, "NULL"), (2, None, "NULL"), (9, None, "NULL"), (12, None, "NULL"),
                         (20, None, "NULL"), (4, None, "cos_cache"), (0, vp(0x10008), "16-byte"), (1, vp(0x18008), "16-byte"),
                         (6, vp(0x18008), "16-byte"), (7, vp(0x18008), "16-byte"), (17, vp(0x88004), "8-byte"),
                         (9, vp(0x38002), "4-byte"), (14, 3, "num_decode_seqs"), (14, -1, "num_decode_seqs"),
                         (3, -1, "num_tokens"), (18, vp(0x100010), "256-byte")]:
        a = list(good)
        a[i] = v
        assert B.lib.pa_quant_mixed(ctypes.byref(_params(B)), *a) == B.PA_ERR_INVALID_ARGUMENT, (i, B.last_error())
        assert needle in B.last_error(), (i, B.last_error())
    a = list(good)
    a[19] = ctypes.c_size_t(16)
    assert B.lib.pa_quant_mixed(ctypes.byref(_params(B)), *a) == B.PA_ERR_WORKSPACE
    assert B.lib.pa_quant_mixed(ctypes.byref(_params(B, cross=1, rotary_dim=0)), *good) == B.PA_ERR_INVALID_ARGUMENT
    good[3] = 0
    assert B.lib.pa_quant_mixed(ctypes.byref(_params(B)), *good) == B.PA_OK


def test_page_tensors_of_whole_pages(B):
    p = B.make_pages_params(num_blocks=8, block_size=16, max_blocks_per_seq=4, num_seqs=4)
    def copy(page_bytes):
        arr = (B.pa_pages_cache * 1)()
        arr[0].data, arr[0].page_bytes = 0x10000, page_bytes
        return B.lib.pa_pages_copy(ctypes.byref(p), arr, 1, _vp(0x20000), _vp(0x30000), None, 0, None,
                                   ctypes.c_size_t(0), None, None)
    for good in (8, 16, 24, 1 << 32, 16 * 16):
        assert copy(B.PA_PAGE_WHOLE | good) == B.PA_OK, B.last_error()
    for bad in (0, 4, 12, (1 << 32) + 8, 1 << 41):
        assert copy(B.PA_PAGE_WHOLE | bad) == B.PA_ERR_INVALID_ARGUMENT
        assert "page_bytes" in B.last_error()


# ---- the oracle

def test_exponents():
    """Against the definition, at and beside every border."""
    for e in range(-60, 60):
        top = math.ldexp(448.0, e)
        for x in (top, np.nextafter(top, 0), np.nextafter(top, np.inf), 0.6 * top):
            got = Q.exponent_for(x)
            fits = [k for k in range(-48, 49) if x <= math.ldexp(448.0, k)]
            assert got == (fits[0] if fits else 48)
    assert Q.exponent_for(0.0) == -48
    assert [Q.stored(x) for x in (1.0, 2.0 ** -48, 2.0 ** 48, 2.0 ** 49, 3.0, -1.0, float("nan"), float("inf"), 0.0)] == \
        [1.0, 2.0 ** -48, 2.0 ** 48, 0, 0, 0, 0, 0, 0]


def test_codes_are_torch_casts():
    x = np.random.default_rng(0).standard_normal(4096) * np.exp(np.random.default_rng(1).standard_normal(4096) * 4)
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (Q.encode(x) == want).all()
    assert Q.encode(np.array([np.nan, np.inf, -np.inf, 1e9, -0.0])).tolist() == [0x7F, 0x7E, 0xFE, 0x7E, 0x80]


def test_writing_in_pieces():
    """A page filled row by row ends with the scale of a single write and codes within the roundings of
    its growth: each time a scale doubles, a code may move by half of its last place."""
    rng = np.random.default_rng(3)
    p = dict(block_size=16, kv_num_heads=2, rotary_dim=0, rotary_offset=0, rotary_interleaved=0, cos_rows=1, rms_eps=0.0)
    key, value = rng.standard_normal((16, 2, 16)) * np.exp(rng.standard_normal((16, 1, 1)) * 2), rng.standard_normal((16, 2, 32))
    key = key.astype(np.float32).astype(np.float64)
    def empty():
        return (np.full((3, 16, 2, 16), 0x7F, np.uint8), np.full((3, 16, 2, 32), 0x55, np.uint8),
                np.full((3, 2, 2), 7.0, np.float32))
    one, many = empty(), empty()
    slots = np.arange(32, 48)
    Q.write(key, value, None, None, slots, [0, 16], [0], *one, p)
    for r in range(16):
        Q.write(key[r:r + 1], value[r:r + 1], None, None, slots[r:r + 1], [0, 1], [r], *many, p)
    assert (one[2][2] == many[2][2]).all() and (one[2][:2] == 7.0).all() and (one[0][:2] == 0x7F).all()
    k1, k2 = (P.e4m3_to_f64(c[0][2]) * c[2][2, :, 0][None, :, None] for c in (one, many))
    assert np.abs(k1 - key).max() <= (np.abs(key) * 2.0 ** -4 + one[2][2, :, 0].max() * 2.0 ** -10).max()
    # the sum of half places of at most 2^-4 relative each (a value below a code's normal range loses more)
    assert (np.abs(k2 - key) <= np.maximum(np.abs(key) * 2.0 ** -3, many[2][2, :, 0][None, :, None] * 2.0 ** -9)).all()


def test_attention_is_the_separate_mode():
    """Over the values the codes stand for, as 16-bit rows do, and cross attention as a window-less read."""
    rng = np.random.default_rng(5)
    p = dict(num_heads=4, kv_num_heads=2, head_size=16, v_head_size=16, block_size=16, rotary_dim=16, rotary_offset=0,
             rotary_interleaved=0, cos_rows=64, scale=0.3, softcap=5.0, local_window_size=9, rms_eps=1e-6, cross=0, dtype=P.BF16)
    kc, vc = (rng.integers(0, 0x78, (6, 16, 2, 16)).astype(np.uint8) for _ in range(2))
    scales = np.ldexp(1.0, rng.integers(-9, -5, (6, 2, 2))).astype(np.float32)
    q = rng.standard_normal((3, 4, 16))
    cos, sin = rng.standard_normal((64, 8)), rng.standard_normal((64, 8))
    cum, past, table = np.array([0, 2, 3]), np.array([20, 5]), np.array([[3, 1], [5, -1]])
    sink, norm = rng.standard_normal(4), rng.standard_normal(16)
    out, _ = Q.attend(q, kc, vc, scales, cos, sin, cum, past, table, p, sink, norm)
    rows = [P.F64Cache((P.e4m3_to_f64(c) * scales[:, None, :, i, None]).reshape(-1, 16)) for i, c in enumerate((kc, vc))]
    for t in range(3):
        want = P.separate_attend_token(t, q[t].reshape(-1), rows[0], rows[1], cos, sin, cum, past, table, p,
                                       head_sink=sink, q_norm=norm)
        np.testing.assert_allclose(out[t], want, rtol=1e-12, atol=1e-14)
    # cross: both tokens of a sequence see its 20 rows; the last of 20 causal tokens does too
    x = dict(p, rotary_dim=0, local_window_size=-1, cross=1)
    out, _ = Q.attend(q, kc, vc, scales, None, None, cum, past, table, x)
    for t, (b, n) in enumerate([(0, 20), (0, 20), (1, 5)]):
        want = P.separate_attend_token(0, q[t].reshape(-1), rows[0], rows[1], None, None, [0, 1], [n - 1], table[b:b + 1],
                                       dict(x))
        np.testing.assert_allclose(out[t], want, rtol=1e-12, atol=1e-14)
    assert not Q.attend(q, kc, vc, scales, None, None, cum, np.array([0, 5]), table, x)[0][:2].any()
