"""Paged caches in 8 bits on the GPU, against the float64 oracle: codes and scales exactly, attention
within the bound that the oracle derives from the roundings."""
import math

import numpy as np
import pytest
import torch

from oracle import pa_oracle as P, quant_oracle as Q

pytestmark = pytest.mark.gpu
DT = {P.BF16: torch.bfloat16, P.F16: torch.float16}


def _api():
    from paged_latent_attention_cache_gb300 import api
    return api


def _binding():
    from paged_latent_attention_cache_gb300 import binding
    return binding


class Case:
    """Sequences of ``q`` new tokens behind ``past`` cached ones (cross: ``past`` encoder rows), pages in
    random order. Rows of the cache that nobody has written hold NaN codes, pages that nobody holds NaN
    scales as well."""

    def __init__(self, q, past, *, dtype=P.BF16, heads=8, kv=2, hs=64, vhs=None, rd=None, ro=0, inter=0, bs=16, window=-1,
                 softcap=0.0, scale=0.0, sink=False, norm=False, cross=0, seed=0, spare=3, gain=1.0, blocks=0, mb=0,
                 stale_nan=True):
        rng = self.rng = np.random.default_rng(seed)
        self.q, self.past = np.array(q), np.array(past)
        vhs = vhs or hs
        rd = (0 if cross else hs) if rd is None else rd
        ctx = self.past if cross else self.q + self.past
        pages = -(-ctx // bs)
        blocks = max(int(pages.sum()) + spare, blocks)
        self.mb = max(int(pages.max(initial=1)), mb, 1)
        self.p = dict(dtype=dtype, num_heads=heads, kv_num_heads=kv, head_size=hs, v_head_size=vhs, rotary_offset=ro,
                      rotary_dim=rd, rotary_interleaved=inter, cos_rows=max(1, int(ctx.max(initial=1))), block_size=bs,
                      num_blocks=blocks, max_blocks_per_seq=self.mb, scale=scale, softcap=softcap,
                      local_window_size=window, rms_eps=1e-5, cross=cross)
        n, T = len(q), int(self.q.sum())
        self.T = T
        perm = rng.permutation(blocks)
        self.table = np.full((n, self.mb), -1, np.int32)
        at = 0
        for b in range(n):
            self.table[b, :pages[b]] = perm[at:at + pages[b]]
            at += pages[b]
        self.cum = np.concatenate([[0], np.cumsum(self.q)]).astype(np.int32)
        r16 = lambda x: P.round_f64(x, dtype)
        cast = self.cast = lambda *s, f=1.0: r16(rng.standard_normal(s) * f)
        self.query = cast(T, heads, hs, f=gain)
        self.key, self.value = cast(T, kv, hs), cast(T, kv, vhs)
        self.key *= np.where(rng.random((T, 1, 1)) < 0.1, 4.0, 1.0)
        ang = np.arange(self.p["cos_rows"])[:, None] * 10000.0 ** (-2.0 * np.arange(rd // 2)[None] / max(rd, 1))
        self.cos, self.sin = r16(np.cos(ang)), r16(np.sin(ang))
        self.sink = cast(heads) if sink else None
        self.q_norm, self.k_norm = (1 + 0.2 * cast(hs), 1 + 0.2 * cast(hs)) if norm else (None, None)
        if norm:
            self.q_norm, self.k_norm = r16(self.q_norm), r16(self.k_norm)
        nan = 0x7F if stale_nan else 0x11
        self.kc, self.vc = (np.full((blocks, bs, kv, w), nan, np.uint8) for w in (hs, vhs))
        self.scales = np.full((blocks, kv, 2), np.nan, np.float32)
        for b in range(n):
            for i in range(pages[b]):
                held = min(bs, int(self.past[b]) - i * bs)
                if held > 0:  # what earlier calls wrote
                    for c, cache in enumerate((self.kc, self.vc)):
                        e = rng.integers(-9, -6, kv)
                        self.scales[self.table[b, i], :, c] = np.ldexp(1.0, e)
                        x = rng.standard_normal((held, kv, cache.shape[3])) * np.ldexp(60.0, 0)
                        cache[self.table[b, i], :held] = Q.encode(x)
        pos = np.concatenate([np.arange(a, a + k) for a, k in zip(self.past, self.q)]) if T else np.zeros(0, int)
        seq = np.repeat(np.arange(n), self.q)
        self.slots = np.full(T, -1, np.int32) if cross else (self.table[seq, pos // bs] * bs + pos % bs).astype(np.int32)

    def dev(self, a, dtype=None):
        t = torch.from_numpy(np.ascontiguousarray(a))
        return t.to("cuda", DT[self.p["dtype"]] if dtype is None else dtype)

    def tensors(self):
        d, i32 = self.dev, torch.int32
        T = self.T
        opt = lambda x: None if x is None else d(x)
        return dict(query=d(self.query).flatten(1), key=d(self.key).flatten(1), value=d(self.value).flatten(1),
                    kc=d(self.kc, torch.uint8), vc=d(self.vc, torch.uint8), scales=d(self.scales, torch.float32),
                    cos=d(self.cos) if self.p["rotary_dim"] else None, sin=d(self.sin) if self.p["rotary_dim"] else None,
                    cum=d(self.cum, i32), past=d(self.past, i32), table=d(self.table, i32), slots=d(self.slots, i32),
                    sink=opt(self.sink), q_norm=opt(self.q_norm), k_norm=opt(self.k_norm))

    def op(self, **kw):
        p = dict(self.p)
        p["dtype"] = DT[p["dtype"]]
        p["cross"] = bool(p["cross"])
        return _api().QuantizedAttention(**p, max_seqs=max(1, len(self.q)), max_tokens=max(1, self.T), **kw)

    def forward(self, op, t, nd, **kw):
        if self.p["cross"]:
            return op.attend(t["query"], t["kc"], t["vc"], t["scales"], None, None, t["cum"], t["past"], t["table"], nd,
                             head_sink=t["sink"], q_norm_weight=t["q_norm"], **kw)
        return op.forward(t["query"], t["key"], t["value"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["cum"],
                          t["past"], t["table"], t["slots"], nd, head_sink=t["sink"], q_norm_weight=t["q_norm"],
                          k_norm_weight=t["k_norm"], **kw)

    def oracle_write(self):
        c = [self.kc.copy(), self.vc.copy(), self.scales.copy()]
        if not self.p["cross"]:
            Q.write(self.key, self.value, self.cos, self.sin, self.slots, self.cum, self.past, *c, self.p, self.k_norm)
        return c

    def oracle(self, caches):
        return Q.attend(self.query, *caches, self.cos, self.sin, self.cum, self.past, self.table, self.p, self.sink,
                        self.q_norm)


def _same_codes(got, want):
    nan = (want & 0x7F) == 0x7F
    assert (((got & 0x7F) == 0x7F) == nan).all()
    assert (got[~nan] == want[~nan]).all(), np.argwhere((got != want) & ~nan)[:5]


def _check_caches(case, t, want):
    for name, w in zip(("kc", "vc"), want):
        _same_codes(t[name].cpu().numpy(), w)
    s = t["scales"].cpu().numpy()
    np.testing.assert_array_equal(s, want[2])


def _check_out(got, want, tol):
    got = got.double().cpu().numpy().reshape(want.shape)
    assert np.isfinite(got).all(), np.argwhere(~np.isfinite(got))[:5]
    over = np.abs(got - want) - tol
    assert (over <= 0).all(), (np.unravel_index(over.argmax(), over.shape), over.max(), np.abs(got - want).max(),
                               float((np.abs(got - want) / np.maximum(tol, 1e-300)).max()))


def _run(case, nd, **kw):
    t, op = case.tensors(), case.op()
    out = case.forward(op, t, nd, **kw)
    assert op.error_flags() == 0
    want = case.oracle_write()
    if case.k_norm is None:
        _check_caches(case, t, want)
    else:  # (the norm's own f32 rounding can tip a code; what attention reads is what is there)
        want = [t["kc"].cpu().numpy(), t["vc"].cpu().numpy(), t["scales"].cpu().numpy()]
    ref, tol = case.oracle(want)
    _check_out(out, ref, tol)
    return out, t, op


# ------------------------------------------------------------------------------------------- write

WRITES = [
    dict(q=[1], past=[0]), dict(q=[1], past=[15]), dict(q=[1], past=[16]), dict(q=[16], past=[0]), dict(q=[17], past=[31]),
    dict(q=[1, 40, 0, 3], past=[5, 0, 9, 30]), dict(q=[100, 64, 1], past=[1, 64, 63], bs=64), dict(q=[300], past=[100], bs=256),
    dict(q=[5, 130], past=[100, 126], bs=128, kv=1, heads=4, hs=128), dict(q=[20, 7], past=[3, 17], hs=80, vhs=48, rd=32, ro=8),
    dict(q=[20, 7], past=[3, 17], hs=256, vhs=256, inter=1), dict(q=[9, 30], past=[17, 0], hs=16, vhs=256, rd=16, kv=8),
    dict(q=[33, 2], past=[0, 50], rd=0, vhs=16), dict(q=[4] * 37, past=list(range(37)), kv=1, heads=1, hs=192, vhs=128, inter=1, rd=64, ro=128),
    # as many threads as pages have rows: 256, and 512 with pages in one piece and in several
    dict(q=[64, 50, 70], past=[0, 20, 63], bs=64, kv=1, heads=1, hs=128), dict(q=[200, 90], past=[5, 0], bs=128, kv=1, heads=1, hs=128, vhs=96),
    dict(q=[300, 280], past=[100, 0], bs=512, kv=1, heads=1, hs=256, inter=1), dict(q=[4000, 1000], past=[60, 10], bs=4096, kv=1, heads=1, hs=16),
]


@pytest.mark.parametrize("dtype", [P.BF16, P.F16])
@pytest.mark.parametrize("kw", WRITES)
def test_write(kw, dtype):
    c = Case(dtype=dtype, **kw)
    t, op = c.tensors(), c.op()
    op.write(t["key"], t["value"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["slots"], t["cum"], t["past"])
    assert op.error_flags() == 0
    _check_caches(c, t, c.oracle_write())


def test_write_many_sequences():
    """More sequences than a CTA looks at in one round, some without tokens."""
    rng = np.random.default_rng(1)
    for n in (128, 129, 2000):
        c = Case(list(rng.integers(0, 3, n)), list(rng.integers(0, 40, n)), kv=1, heads=1, hs=16, vhs=16)
        t, op = c.tensors(), c.op()
        op.write(t["key"], t["value"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["slots"], t["cum"], t["past"])
        assert op.error_flags() == 0
        _check_caches(c, t, c.oracle_write())


@pytest.mark.parametrize("kw", [dict(bs=64, hs=128), dict(bs=128, hs=64, vhs=256, inter=1), dict(bs=256, hs=32, rd=0), dict(bs=16, hs=256)])
def test_write_long_among_many_short(kw):
    """Full pages in pieces beside single tokens: NaN and infinities in one piece and not in the others."""
    n = 700
    c = Case([1] * n + [300, 70, 2], list(range(n)) + [5, 0, 62], kv=2, heads=2, seed=47, **kw)
    c.value[n + 130, 0, 3], c.value[n + 131, 1, 4], c.key[n + 250, 1, -1] = np.inf, np.nan, np.nan
    t, op = c.tensors(), c.op()
    op.write(t["key"], t["value"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["slots"], t["cum"], t["past"])
    assert op.error_flags() == 0
    _check_caches(c, t, c.oracle_write())


def test_write_borders_and_extremes():
    """Magnitudes at and beside 448 * 2^e, zeros, subnormals, the largest values, infinities and NaN."""
    for dtype in (P.BF16, P.F16):
        c = Case([16] * 12, [0] * 12, dtype=dtype, kv=1, heads=1, rd=0, seed=4)
        big = 65504.0 if dtype == P.F16 else 3.0e38
        tops = [448.0, 448.0 * 2 ** -7, 452.0, 450.0, 0.0, 2.0 ** -24, big, 2.0 ** -14, 1.0, 447.0, np.inf, np.nan]
        for i, top in enumerate(tops):
            rows = slice(16 * i, 16 * i + 16)
            m = abs(top) if np.isfinite(top) else 3.0
            for x in (c.key, c.value):
                x[rows] = P.round_f64(np.clip(x[rows], -1, 1) * m, dtype)
                x[16 * i + 5, 0, 3], x[16 * i + 6, 0, 7] = top, -top
        t, op = c.tensors(), c.op()
        op.write(t["key"], t["value"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["slots"], t["cum"], t["past"])
        assert op.error_flags() == 0
        _check_caches(c, t, c.oracle_write())


def test_write_in_pieces_and_over():
    """A page filled token by token, then overwritten from the middle and from row 0."""
    c = Case([48], [0], kv=2, seed=5)
    c.key *= np.exp(np.random.default_rng(0).standard_normal((48, 1, 1)) * 2)
    c.key = P.round_f64(c.key, P.BF16)
    t, op = c.tensors(), c.op()
    want = [c.kc.copy(), c.vc.copy(), c.scales.copy()]
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    def step(a, b):
        past = torch.tensor([a], dtype=torch.int32, device="cuda")
        cum = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        op.write(t["key"][a:b].contiguous(), t["value"][a:b].contiguous(), t["kc"], t["vc"], t["scales"], t["cos"],
                 t["sin"], t["slots"][a:b].contiguous(), cum, past)
        Q.write(c.key[a:b], c.value[a:b], c.cos, c.sin, c.slots[a:b], [0, b - a], [a], *want, c.p)
        _check_caches(c, t, want)
    for a in range(20):
        step(a, a + 1)
    for a, b in ((7, 12), (16, 30), (30, 48), (0, 3), (1, 2)):
        step(a, b)
    assert op.error_flags() == 0


def test_write_skips_and_refusals():
    """Slots of -1 leave their rows to grow with the page; slots that break the rules are skipped and told."""
    B = _binding()
    c = Case([30, 20], [5, 0], seed=6)
    good = c.slots.copy()
    c.slots[[3, 11, 35]] = -1
    t, op = c.tensors(), c.op()
    args = lambda: (t["key"], t["value"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["slots"], t["cum"], t["past"])
    op.write(*args())
    assert op.error_flags() == 0
    _check_caches(c, t, c.oracle_write())
    for slot in (good[8] + 1, c.p["num_blocks"] * 16 + int(good[8]) % 16, -2, int(good[25]) // 16 * 16 + int(good[8]) % 16):
        c.slots = good.copy()
        c.slots[8] = slot
        t, op = c.tensors(), c.op()
        op.write(*args())
        assert op.error_flags() == B.PA_DEVERR_SLOT
        if slot // 16 != good[25] // 16:  # (that row of the other page belongs to another token too)
            _check_caches(c, t, c.oracle_write())
    c.slots = good.copy()
    c.p["cos_rows"] = 20
    t, op = c.tensors(), c.op()
    op.write(*args())
    assert op.error_flags() == B.PA_DEVERR_POSITION
    _check_caches(c, t, c.oracle_write())


def test_write_bad_offsets():
    B = _binding()
    c = Case([6, 5], [0, 3], seed=7)
    for cum, past, flag in ([[0, 6, 10], [0, 3], B.PA_DEVERR_CUMSEQ], [[0, 6, 12], [0, 3], B.PA_DEVERR_CUMSEQ],
                            [[0, 7, 5], [0, 3], B.PA_DEVERR_CUMSEQ], [[1, 6, 11], [0, 3], B.PA_DEVERR_CUMSEQ],
                            [[0, 6, 11], [-1, 3], B.PA_DEVERR_CONTEXT], [[-5, 6, 11], [0, 3], B.PA_DEVERR_CUMSEQ]):
        t, op = c.tensors(), c.op()
        t["cum"], t["past"] = c.dev(cum, torch.int32), c.dev(past, torch.int32)
        op.write(t["key"], t["value"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["slots"], t["cum"], t["past"])
        assert op.error_flags() & flag, (cum, op.error_flags())


def test_write_with_norm():
    """The norm in f32: every code is the nearest of a value within 2^-20 of the oracle's."""
    c = Case([33, 20], [0, 9], norm=True, seed=8)
    t, op = c.tensors(), c.op()
    op.write(t["key"], t["value"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["slots"], t["cum"], t["past"],
             k_norm_weight=t["k_norm"])
    want = c.oracle_write()
    np.testing.assert_array_equal(t["scales"].cpu().numpy(), want[2])
    _same_codes(t["vc"].cpu().numpy(), want[1])
    got, ref = P.e4m3_to_f64(t["kc"].cpu().numpy()), P.e4m3_to_f64(want[0])
    ok = np.isnan(ref) | (np.abs(got - ref) <= np.maximum(np.abs(ref) * 2.0 ** -3, 2.0 ** -9))  # a neighbour
    assert ok.all() and (np.isnan(ref) | (got == ref)).mean() > 0.999


# ----------------------------------------------------------------------------------------- restore

@pytest.mark.parametrize("dtype", [P.BF16, P.F16])
@pytest.mark.parametrize("kw", WRITES[:12])
def test_restore(kw, dtype):
    c = Case(dtype=dtype, **kw)
    t, op = c.tensors(), c.op()
    op.write(t["key"], t["value"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["slots"], t["cum"], t["past"])
    k, v = op.restore(t["kc"], t["vc"], t["scales"], t["cum"], t["past"], t["table"], c.T)
    assert op.error_flags() == 0
    want = c.oracle_write()
    top = 65504.0 if dtype == P.F16 else np.inf
    for got, cache, i in ((k, want[0], 0), (v, want[1], 1)):
        x = P.e4m3_to_f64(cache.reshape(-1, *cache.shape[2:])[c.slots]) * want[2][c.slots // c.p["block_size"], :, i][..., None]
        x = P.round_f64(np.clip(x, -top, top), dtype)
        assert (got.double().cpu().numpy().reshape(x.shape) == x).all()


def test_restore_any_range_and_errors():
    B = _binding()
    c = Case([1, 1, 1], [70, 40, 33], seed=9)
    t, op = c.tensors(), c.op()
    cum, past = c.dev([0, 50, 50, 60], torch.int32), c.dev([20, 0, 3], torch.int32)
    k, v = op.restore(t["kc"], t["vc"], t["scales"], cum, past, t["table"], 60)
    assert op.error_flags() == 0
    for i, (b, pos) in enumerate([(0, 20 + i) for i in range(50)] + [(2, 3 + i) for i in range(10)]):
        page, row = c.table[b, pos // 16], pos % 16
        x = P.e4m3_to_f64(c.vc[page, row]) * c.scales[page, :, 1][:, None]
        assert (v[i].double().cpu().numpy() == x.reshape(-1)).all()
    key = torch.full((70, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    value = key.clone()
    op.restore(t["kc"], t["vc"], t["scales"], cum, past, t["table"], 70, key=key, value=value)
    assert op.error_flags() == B.PA_DEVERR_CUMSEQ and bool((key[60:] == 7).all()) and bool((key[:60] == k).all())
    op.reset_error_flags()
    t["table"][0, 2] = c.p["num_blocks"]
    k2, _ = op.restore(t["kc"], t["vc"], t["scales"], cum, past, t["table"], 60)
    assert op.error_flags() == B.PA_DEVERR_BLOCK
    gone = [i for i in range(50) if (20 + i) // 16 == 2]
    assert not k2[gone].any() and bool((k2[50:] == k[50:]).all())
    op.reset_error_flags()
    op.restore(t["kc"], t["vc"], t["scales"], c.dev([0, 50], torch.int32), c.dev([c.mb * 16 - 10], torch.int32),
               t["table"][1:2].contiguous(), 50)
    assert op.error_flags() & B.PA_DEVERR_CONTEXT


@pytest.mark.parametrize("dtype", [P.BF16, P.F16])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("none", [0.0, -0.0, 3.0, -1.0, 2.0 ** 49, math.inf, math.nan])
def test_pages_without_a_scale_are_zeros(none, which, dtype):
    """Whatever their codes, NaN among them: read back, in decode and in prefill of few and of many tokens. The
    other cache's rows of the page, which have a scale, and the pages beside it keep theirs."""
    for q, nd in (([1, 1], 2), ([3, 2], 0), ([40, 30], 0)):
        c = Case(q, [100, 90], dtype=dtype, rd=0, seed=44)
        t, op = c.tensors(), c.op()
        op.write(t["key"], t["value"], t["kc"], t["vc"], t["scales"], None, None, t["slots"], t["cum"], t["past"])
        page = int(c.table[0, 2])
        cache = t["vc" if which else "kc"]
        t["scales"][page, :, which] = none
        cache[page] = 0x7F
        cum, past = c.dev([0, 100, 190], torch.int32), c.dev([0, 0], torch.int32)
        read = lambda: [*op.restore(t["kc"], t["vc"], t["scales"], cum, past, t["table"], 190),
                        op.attend(t["query"], t["kc"], t["vc"], t["scales"], None, None, t["cum"], t["past"], t["table"], nd)]
        got = read()
        assert op.error_flags() == 0
        assert not got[which][32:48].any()
        cache[page] = 0
        t["scales"][page, :, which] = 1.0
        want = read()
        assert all(torch.equal(a, b) and torch.isfinite(a).all() for a, b in zip(got[:2], want[:2]))
        # (a page's scale of nothing is the least one in the values' exponents: other roundings)
        assert torch.isfinite(got[2]).all()
        caches = [t["kc"].cpu().numpy(), t["vc"].cpu().numpy(), t["scales"].cpu().numpy()]
        _check_out(got[2], *c.oracle(caches))


# --------------------------------------------------------------------------------------- attention

DECODES = [
    dict(q=[1], past=[0]), dict(q=[1], past=[14]), dict(q=[1, 1, 1], past=[15, 16, 17]), dict(q=[1] * 5, past=[0, 1, 100, 255, 256]),
    dict(q=[1, 1], past=[2000, 3], bs=64), dict(q=[1, 1], past=[700, 900], heads=8, kv=8), dict(q=[1, 1], past=[700, 900], heads=3, kv=1),
    dict(q=[1, 1], past=[300, 90], heads=32, kv=2), dict(q=[1, 1], past=[300, 90], heads=20, kv=1), dict(q=[1, 1], past=[200, 90], heads=128, kv=1),
    dict(q=[1, 1], past=[300, 333], hs=128), dict(q=[1, 1], past=[300, 333], hs=256, vhs=256), dict(q=[1, 1], past=[300, 333], hs=192, vhs=128, heads=32, kv=2),
    dict(q=[1, 1], past=[100, 333], hs=80, vhs=48, rd=32, ro=16), dict(q=[1, 1], past=[100, 333], hs=16, vhs=16),
    dict(q=[1, 1], past=[100, 333], hs=96, vhs=96, inter=1), dict(q=[1, 1], past=[100, 333], hs=64, vhs=256, heads=28, kv=4),
    dict(q=[1, 1, 1], past=[500, 40, 77], window=33), dict(q=[1, 1], past=[500, 40], window=0), dict(q=[1, 1], past=[500, 40], window=127, bs=64),
    dict(q=[1, 1], past=[500, 40], softcap=3.0, sink=True), dict(q=[1, 1], past=[500, 40], norm=True, sink=True),
    dict(q=[1, 1], past=[500, 40], scale=2.0, gain=8.0), dict(q=[1, 1], past=[3000, 4000], bs=128, heads=2, kv=1, hs=128),
]


@pytest.mark.parametrize("dtype", [P.BF16, P.F16])
@pytest.mark.parametrize("kw", DECODES)
def test_decode(kw, dtype):
    _run(Case(dtype=dtype, **kw), len(kw["q"]))


@pytest.mark.parametrize("softcap", [0.3, 128.0, 129.0, 3e2, 1e4, 1e6, 1e9, 1e18, 2e18, 3e38])
@pytest.mark.parametrize("q", [[1, 1], [3, 2], [60, 9]])
def test_softcaps_of_any_size(q, softcap):
    """One far above the scores leaves them as they are, one below them all but decides them. (Some outputs are
    below 2^-14, where fp16 values are 2^-24 apart and rounding moves one by up to 2^-25.)"""
    for kw in (dict(), dict(hs=256, vhs=256)):
        c = Case(q, [400, 90], dtype=P.F16, softcap=softcap, gain=4.0, seed=52, **kw)
        t, op = c.tensors(), c.op()
        out = c.forward(op, t, 2 if q == [1, 1] else 0)
        assert op.error_flags() == 0
        want = c.oracle_write()
        _check_caches(c, t, want)
        ref, tol = c.oracle(want)
        _check_out(out, ref, tol + 2.0 ** -25)


PREFILLS = [
    dict(q=[1], past=[0]), dict(q=[2], past=[0]), dict(q=[3, 1, 0, 5], past=[0, 30, 7, 16]), dict(q=[130], past=[0]),
    dict(q=[70, 20], past=[100, 300], bs=64), dict(q=[129, 64], past=[127, 0], heads=4, kv=4), dict(q=[40, 30], past=[90, 0], heads=3, kv=1),
    dict(q=[7, 30], past=[90, 0], heads=64, kv=2), dict(q=[5, 9], past=[90, 200], heads=128, kv=1), dict(q=[20, 9], past=[90, 200], heads=10, kv=2),
    dict(q=[60, 9], past=[90, 200], hs=128), dict(q=[60, 9], past=[90, 200], hs=128, heads=8, kv=8, bs=128), dict(q=[60, 9], past=[90, 200], hs=256, vhs=256),
    dict(q=[60, 9], past=[90, 200], hs=192, vhs=128), dict(q=[60, 9], past=[90, 200], hs=80, vhs=48, rd=32, ro=16),
    dict(q=[60, 9], past=[90, 200], hs=16, vhs=16), dict(q=[60, 9], past=[90, 200], hs=64, vhs=256, inter=1),
    dict(q=[100, 9], past=[90, 300], window=20), dict(q=[100, 9], past=[90, 300], window=0), dict(q=[200], past=[300], window=150, bs=64, heads=2, kv=1),
    dict(q=[60, 9], past=[90, 200], softcap=3.0, sink=True), dict(q=[60, 9], past=[90, 200], norm=True, sink=True),
    dict(q=[60, 9], past=[90, 200], scale=2.0, gain=8.0), dict(q=[300, 3], past=[400, 2000], heads=2, kv=1, bs=32),
    dict(q=[4, 6], past=[2500, 3100], heads=8, kv=2, bs=64, hs=128),
]


@pytest.mark.parametrize("dtype", [P.BF16, P.F16])
@pytest.mark.parametrize("kw", PREFILLS)
def test_prefill(kw, dtype):
    _run(Case(dtype=dtype, **kw), 0)


@pytest.mark.parametrize("kw,nd", [
    (dict(q=[1, 1, 1], past=[0, 5, 300]), 3), (dict(q=[1, 1], past=[33, 1000], heads=8, kv=8, bs=64), 2),
    (dict(q=[1, 1], past=[33, 100], sink=True, softcap=4.0), 2), (dict(q=[40, 7], past=[100, 0]), 0),
    (dict(q=[300, 2, 0, 1], past=[77, 1, 50, 129], bs=64, heads=4, kv=4), 0), (dict(q=[1, 30], past=[90, 90], hs=128, norm=True), 1),
    (dict(q=[5, 600], past=[2000, 17], heads=2, kv=2), 0)])
def test_cross(kw, nd):
    c = Case(cross=1, seed=11, **kw)
    out, _, _ = _run(c, nd)
    for b in range(len(c.q)):
        if c.past[b] == 0:
            assert not out[c.cum[b]:c.cum[b + 1]].any()


def test_cross_after_its_write():
    """An encoder's states written as tokens of their sequence, then read by every decoder step."""
    c = Case([37, 100, 3], [0, 0, 0], rd=0, seed=12)
    t, writer = c.tensors(), c.op()
    writer.write(t["key"], t["value"], t["kc"], t["vc"], t["scales"], None, None, t["slots"], t["cum"], t["past"])
    caches = c.oracle_write()
    _check_caches(c, t, caches)
    p = dict(c.p, cross=1)
    for q in ([1, 1, 1], [4, 1, 30]):
        query = c.cast(sum(q), 8, 64)
        cum = np.concatenate([[0], np.cumsum(q)])
        kw = dict(p, dtype=torch.bfloat16, cross=True)
        op = _api().QuantizedAttention(**kw, max_seqs=3, max_tokens=64)
        out = op.attend(c.dev(query).view(sum(q), -1), t["kc"], t["vc"], t["scales"], None, None, c.dev(cum, torch.int32),
                        c.dev(c.q, torch.int32), t["table"], 3 if max(q) == 1 else 0)
        assert op.error_flags() == 0
        ref, tol = Q.attend(query, *caches, None, None, cum, c.q, c.table, p)
        _check_out(out, ref, tol)


def test_one_call_is_three():
    """forward against write, decode and prefill by themselves."""
    c = Case([1, 1, 40, 2], [10, 300, 64, 20], sink=True, norm=True, seed=28)
    t, op = c.tensors(), c.op()
    want = c.forward(op, t, 2)
    t, out = c.tensors(), torch.empty_like(want)
    op.write(t["key"], t["value"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["slots"], t["cum"], t["past"],
             k_norm_weight=t["k_norm"])
    args = (t["query"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["cum"], t["past"], t["table"], out)
    op.decode(*args, 0, 2, head_sink=t["sink"], q_norm_weight=t["q_norm"], after_write=True)
    op.prefill(*args, 2, 4, head_sink=t["sink"], q_norm_weight=t["q_norm"])
    assert op.error_flags() == 0 and torch.equal(out, want)


@pytest.mark.parametrize("q,past,kw", [
    ([1] * 6, [3000] * 6, dict(heads=8, kv=2)), ([1] * 4, [2500] * 4, dict(heads=16, kv=1, hs=128)),
    ([1] * 6, [2000] * 6, dict(heads=8, kv=2, hs=192, vhs=128)), ([2] * 3, [1500] * 3, dict(heads=16, kv=2, hs=256)),
    ([70], [3000], dict(heads=4, kv=2)), ([65, 30], [1000, 2500], dict(heads=8, kv=2, hs=128)),
    ([70], [2000], dict(heads=4, kv=2, hs=176, vhs=96)), ([70], [1000], dict(heads=4, kv=2, hs=256)),
    ([70], [1000], dict(heads=4, kv=2, hs=256, vhs=64)), ([70], [1000], dict(heads=4, kv=2, hs=80, vhs=144)),
    ([70], [2000], dict(heads=4, kv=2, rd=0, norm=True)), ([1] * 6, [3000] * 6, dict(heads=8, kv=2, rd=0, norm=True))])
def test_fp16_keeps_its_bits(q, past, kw):
    """Rotated and normalized queries keep more than fp16 holds. A rounding to fp16 is 2^-11 sqrt(0.541 / 3) =
    2.07e-4 off in the 2-norm, 0.541 being the mean of 1 / m^2 over mantissas m in [1, 2) spread evenly in their
    logarithm. The probabilities' and the output's own are allowed: 2.93e-4 together, and an eighth more for chance
    (some 256 rows and more). A third one in the query, where scores spread by 1 or more, makes it 3.6e-4."""
    c = Case(q, past, dtype=P.F16, bs=64, gain=4.0, seed=3, **kw)
    t, op = c.tensors(), c.op()
    out = c.forward(op, t, len(q) if max(q) == 1 else 0)
    assert op.error_flags() == 0
    want = c.oracle([t["kc"].cpu().numpy(), t["vc"].cpu().numpy(), t["scales"].cpu().numpy()])[0]
    off = out.double().cpu().numpy().reshape(want.shape) - want
    assert np.linalg.norm(off) < 3.3e-4 * np.linalg.norm(want), np.linalg.norm(off) / np.linalg.norm(want)


def test_own_slots_with_a_page_that_grows():
    """The promise changes no result, also where the call's rows rescale what is read below them."""
    for q, nd in (([1, 1, 1], 3), ([40, 3, 70], 0)):
        c = Case(q, [200, 77, 20], bs=64, seed=51)
        c.key *= 64.0
        c.value *= 64.0
        t, op = c.tensors(), c.op()
        want = c.forward(op, t, nd)
        for own in (False, True):
            t, op = c.tensors(), c.op(own_slots=own)
            before = t["scales"].clone()
            op.write(t["key"], t["value"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["slots"], t["cum"], t["past"])
            out = torch.empty_like(want)
            (op.decode if nd else op.prefill)(t["query"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["cum"],
                                              t["past"], t["table"], out, after_write=True)
            assert op.error_flags() == 0 and torch.equal(out, want)
            page = int(c.table[0, 3])
            assert bool((t["scales"][page] > before[page]).all())


def test_mixed_batch():
    c = Case([1, 1, 1, 50, 9], [10, 300, 64, 20, 0], sink=True, seed=13)
    _run(c, 3)


@pytest.mark.parametrize("q,past,kw", [
    ([5, 3, 4, 5], [2000, 500, 33, 1000], dict(heads=8, kv=2, hs=128)), ([200], [1500], dict(heads=8, kv=2)),
    ([70, 20], [700, 1200], dict(heads=4, kv=1, dtype=P.F16)), ([1, 2], [900, 40], dict(heads=16, kv=2)),
    ([60], [900], dict(heads=4, kv=2, hs=256, vhs=256))])
def test_a_range_does_not_depend_on_what_stands_beside_it(q, past, kw):
    """Prefill sequences beside many decode sequences take the same way, bit for bit, as by themselves."""
    nd = 120
    c = Case([1] * nd + q, list(range(nd)) + past, bs=64, seed=45, **kw)
    t, op = c.tensors(), c.op()
    op.write(t["key"], t["value"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["slots"], t["cum"], t["past"])
    out = op.attend(t["query"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["cum"], t["past"], t["table"], nd)
    alone = op.attend(t["query"][nd:].contiguous(), t["kc"], t["vc"], t["scales"], t["cos"], t["sin"],
                      t["cum"][nd:] - nd, t["past"][nd:].contiguous(), t["table"][nd:].contiguous(), 0)
    assert op.error_flags() == 0
    _check_out(out, *c.oracle([t["kc"].cpu().numpy(), t["vc"].cpu().numpy(), t["scales"].cpu().numpy()]))
    assert torch.equal(out[nd:], alone)


@pytest.mark.parametrize("q", [[3, 4], [150, 40], [600]])
def test_a_range_among_sequences_without_tokens(q):
    """More tokens than the others' number makes likely: rows outside the range stay, all of it is there."""
    n = 300
    c = Case([0] * n + q + [0] * n, [0] * n + [400, 70][:len(q)] + [0] * n, heads=4, kv=2, bs=64, seed=46)
    t, op = c.tensors(), c.op()
    op.write(t["key"], t["value"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["slots"], t["cum"], t["past"])
    want = c.oracle([t["kc"].cpu().numpy(), t["vc"].cpu().numpy(), t["scales"].cpu().numpy()])
    out = torch.full((c.T, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    args = (t["query"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["cum"], t["past"], t["table"], out)
    op.prefill(*args, n, n + len(q))
    assert op.error_flags() == 0
    _check_out(out, *want)
    out.fill_(7.0)
    op.prefill(*args, n + len(q) - 1, n + len(q))
    first = c.T - q[-1]
    assert op.error_flags() == 0 and bool((out[:first] == 7).all())
    _check_out(out[first:], want[0][first:], want[1][first:])


SKEWED = [  # few rows on average: 1 and 300 tokens, and sequences of 1024 rows and a token more
    dict(q=[1] * 100 + [300] + [1] * 20, past=list(range(100)) + [600] + [7] * 20, heads=8, kv=1),
    dict(q=[0, 3] * 120 + [256, 257] + [2] * 60, past=[5, 90] * 120 + [0, 300] + [64] * 60, heads=4, kv=1, bs=64, sink=True),
    dict(q=[400] + [1] * 90, past=[100] + [30] * 90, heads=16, kv=2, window=50, softcap=8.0),
    dict(q=[1] * 90 + [150], past=[40] * 90 + [0], heads=16, kv=1, hs=256, vhs=256, inter=1, norm=True),
]


@pytest.mark.parametrize("dtype", [P.BF16, P.F16])
@pytest.mark.parametrize("kw", SKEWED)
def test_long_sequences_among_short_ones(kw, dtype):
    _run(Case(dtype=dtype, seed=48, **kw), 0)


def test_long_and_short_sequences_tell_their_errors():
    """Each kernel tells of its own sequences, and the others keep their results."""
    B = _binding()
    c = Case([1] * 100 + [300] + [1] * 20, list(range(100)) + [600] + [7] * 20, heads=8, kv=1, seed=49)
    op, t = c.op(), c.tensors()
    op.write(t["key"], t["value"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["slots"], t["cum"], t["past"])
    ref, tol = c.oracle(c.oracle_write())
    rows = lambda b: slice(int(c.cum[b]), int(c.cum[b + 1]))
    assert c.cum[101] == 400

    def run(change):
        x = {k: v.clone() if v is not None else None for k, v in t.items()}
        change(x)
        op.reset_error_flags()
        out = torch.full((c.T, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        op.attend(x["query"], x["kc"], x["vc"], x["scales"], x["cos"], x["sin"], x["cum"], x["past"], x["table"], 0, out=out)
        return out, op.error_flags()

    def others(out, gone):
        keep = np.ones(c.T, bool)
        keep[rows(gone)] = False
        _check_out(out[torch.from_numpy(keep).cuda()], ref[keep], tol[keep])

    for b, page in ((99, 0), (100, 2)):  # a short one, the long one
        for bad in (-1, c.p["num_blocks"]):
            out, flags = run(lambda x: x["table"][b, page].fill_(bad))
            assert flags == B.PA_DEVERR_BLOCK and not out[rows(b)].any()
            if b == 100:
                others(out, b)
        for past in (-1, c.mb * 16, 2 ** 31 - 1):
            out, flags = run(lambda x: x["past"][b].fill_(past))
            assert flags == B.PA_DEVERR_CONTEXT and not out[rows(b)].any()
            others(out, b)
    for at, value in ((101, c.T + 1), (100, 2 ** 31 - 1), (0, -5), (0, -(2 ** 31)), (100, 500)):
        out, flags = run(lambda x: x["cum"][at].fill_(value))
        assert flags & B.PA_DEVERR_CUMSEQ


def test_long_and_short_sequences_captured():
    c = Case([1] * 100 + [300] + [1] * 20, list(range(100)) + [600] + [7] * 20, heads=8, kv=1, seed=50)
    t, op = c.tensors(), c.op()
    want = c.forward(op, t, 0).clone()
    assert torch.equal(c.forward(op, t, 0), want)
    t2, out = c.tensors(), torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.forward(op, t2, 0, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_scales_apart():
    """Pages whose scales lie far apart: values of 2^-48 .. 2^40 in one row's keys, and empty pages of
    zeros among them."""
    for nd, q in ((2, [1, 1]), (0, [40, 20])):
        c = Case(q, [200, 160], rd=0, heads=4, kv=2, seed=14, window=-1)
        rng = np.random.default_rng(2)
        held = np.unique(c.table[c.table >= 0])
        for g in range(2):
            c.scales[held, g, 1] = np.ldexp(1.0, rng.choice([-48, -30, -9, -8, 0, 20], len(held)))
            c.scales[held, g, 0] = np.ldexp(1.0, rng.choice([-48, -12, -9, -8], len(held)))
        c.vc[held[::3]] = 0
        c.kc[held[1::4]] = 0
        c.vc[(c.vc & 0x7F) == 0x7F] = 0x30
        c.kc[(c.kc & 0x7F) == 0x7F] = 0x30
        _run(c, nd)


def test_one_key_takes_nearly_all():
    """A key with nearly all of the weight and a value near zero: the others' parts survive."""
    for small in (2.0 ** -12, 2.0 ** -20):
        for nd, q in ((1, [1]), (0, [5])):
            c = Case(q, [250], rd=0, heads=4, kv=2, seed=15, dtype=P.F16)
            c.query = P.round_f64(np.abs(c.query) + 0.5, P.F16)
            page, row = c.table[0, 3], 5
            held = c.table[0][c.table[0] >= 0]
            c.scales[held, :, 0] = 2.0 ** -9
            c.scales[held, :, 1] = 2.0 ** -7
            c.kc[page, row] = Q.encode(np.array(60.0 + 0.0))  # q . K large
            c.p["scale"] = float(-np.log(small) / (c.query.sum(-1).mean() * 60.0 * 2.0 ** -9))
            c.vc[page, row] = 0
            _run(c, nd)


# ------------------------------------------------------------------ masked places, errors, untouched rows

def test_nan_seen_and_unseen():
    """A NaN value or key reaches the rows that see it and no others."""
    for what in ("vc", "kc"):
        c = Case([70], [40], rd=0, heads=2, kv=1, seed=16, stale_nan=True)
        x = c.value if what == "vc" else c.key
        x[33, 0, 5] = np.nan  # position 73
        t, op = c.tensors(), c.op()
        out = c.forward(op, t, 0).double().cpu().numpy().reshape(70, 2, 64)
        assert np.isfinite(out[:33]).all() and np.isnan(out[33:]).any((1, 2)).all()
        c.key[33], c.value[33] = 1.0, 1.0
        ref, tol = c.oracle(c.oracle_write())
        assert (np.abs(out[:33] - ref[:33]) <= tol[:33]).all()
        # behind a window again
        c = Case([70], [40], rd=0, heads=2, kv=1, seed=16, window=10)
        (c.value if what == "vc" else c.key)[33, 0, 5] = np.nan
        t, op = c.tensors(), c.op()
        out = c.forward(op, t, 0).double().cpu().numpy().reshape(70, 2, 64)
        bad = np.isnan(out).any((1, 2))
        assert bad[33:44].all() and not bad[:33].any() and not bad[44:].any()


def test_pages_without_scales():
    """Rows of a page that has no scale count as zeros."""
    c = Case([1, 1], [100, 90], rd=0, seed=17)
    c.scales[c.table[0, 2]] = 0.0
    c.scales[c.table[1, 1], :, 1] = 3.0
    _run(c, 2)
    _run(c, 0)


def test_error_flags_and_rows():
    B = _binding()
    for nd in (3, 0):
        c = Case([1, 1, 1], [100, 90, 5], seed=18)
        ref, tol = c.oracle(c.oracle_write())
        full = lambda t: torch.full((t["query"].size(0), 512), 7.0, dtype=torch.bfloat16, device="cuda")
        t, op = c.tensors(), c.op()
        t["table"][1, 2] = -1  # an invalid page among what is read
        out = full(t)
        c.forward(op, t, nd, out=out)
        assert op.error_flags() == B.PA_DEVERR_BLOCK
        assert not out[1].any()
        _check_out(out[[0, 2]], ref[[0, 2]], tol[[0, 2]])
        # positions beyond the table
        t, op = c.tensors(), c.op()
        t["past"][0] = c.mb * 16
        out = full(t)
        op.attend(t["query"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["cum"], t["past"], t["table"], nd, out=out)
        assert op.error_flags() & B.PA_DEVERR_CONTEXT and not out[0].any()
        t["past"][0] = -1
        op.reset_error_flags()
        op.attend(t["query"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["cum"], t["past"], t["table"], nd, out=out)
        assert op.error_flags() & B.PA_DEVERR_CONTEXT and not out[0].any()
        # beyond the rotary table
        c2 = Case([1, 1, 1], [100, 90, 5], seed=18)
        c2.p["cos_rows"] = 95
        t, op = c2.tensors(), c2.op()
        out = full(t)
        op.attend(t["query"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["cum"], t["past"], t["table"], nd, out=out)
        assert op.error_flags() & B.PA_DEVERR_POSITION and not out[0].any()
    # a decode sequence with two new tokens: told, rows as they were
    c = Case([1, 2, 1], [20, 30, 40], seed=19)
    t, op = c.tensors(), c.op()
    out = torch.full((4, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    c.forward(op, t, 3, out=out)
    assert op.error_flags() == B.PA_DEVERR_DECODE_QLEN and bool((out[1:3] == 7).all())
    ref, tol = c.oracle(c.oracle_write())
    _check_out(out[[0, 3]], ref[[0, 3]], tol[[0, 3]])


@pytest.mark.parametrize("vhs", [64, 256])
def test_error_flags_of_long_prefill(vhs):
    """As above, in sequences of many tokens (a kernel of its own): the others keep their results."""
    B = _binding()
    c = Case([60, 90, 40], [100, 300, 5], vhs=vhs, seed=31)
    ref, tol = c.oracle(c.oracle_write())
    want = lambda s: (ref[s], tol[s])

    def run(change):
        t, op = c.tensors(), c.op()
        op.write(t["key"], t["value"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["slots"], t["cum"], t["past"])
        change(t)
        out = torch.full((c.T, 8 * vhs), 7.0, dtype=torch.bfloat16, device="cuda")
        op.attend(t["query"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["cum"], t["past"], t["table"], 0, out=out)
        return out, op.error_flags()

    out, flags = run(lambda t: t["table"][1, 2].fill_(-1))
    assert flags == B.PA_DEVERR_BLOCK and not out[60:150].any()
    out, flags = run(lambda t: t["table"][1, 2].fill_(c.p["num_blocks"]))
    assert flags == B.PA_DEVERR_BLOCK and not out[60:150].any()
    _check_out(out[:60], *want(slice(0, 60)))
    _check_out(out[150:], *want(slice(150, 190)))
    for past in (c.mb * 16, -1, -(2 ** 31), 2 ** 31 - 1):
        out, flags = run(lambda t: t["past"][0].fill_(past))
        assert flags & B.PA_DEVERR_CONTEXT and not out[:60].any()
        _check_out(out[60:], *want(slice(60, 190)))
    for cum in ([0, 60, 40, 190], [0, 60, 150, 150], [0, 0, 0, 190]):  # (in bounds, whatever they say)
        out, flags = run(lambda t: t["cum"].copy_(torch.tensor(cum, dtype=torch.int32)))
        assert bool(flags & B.PA_DEVERR_CUMSEQ) == (cum[2] < cum[1])
        assert torch.isfinite(out.float()).all()
    for cum in ([0, 60, 150, 191], [0, 60, 2 ** 31 - 1, 190], [-5, 60, 150, 190], [-(2 ** 31), 60, 150, 190]):
        out, flags = run(lambda t: t["cum"].copy_(torch.tensor(cum, dtype=torch.int32)))
        assert flags & B.PA_DEVERR_CUMSEQ


def test_offsets_that_do_not_rise():
    """Reads of few tokens: told, and nothing out of place."""
    B = _binding()
    c = Case([1] * 6, [40, 3, 0, 100, 64, 9], seed=32)
    for cum in ([0, 1, 5, 3, 4, 5, 6], [0, 1, 2, 7, 4, 5, 6], [-1, 1, 2, 3, 4, 5, 6], [0, 2 ** 31 - 1, -(2 ** 31), 3, 4, 5, 6]):
        for nd in (0, 6):
            t, op = c.tensors(), c.op()
            t["cum"].copy_(torch.tensor(cum, dtype=torch.int32))
            out = torch.full((6, 512), 7.0, dtype=torch.bfloat16, device="cuda")
            c.forward(op, t, nd, out=out)
            assert op.error_flags() & (B.PA_DEVERR_CUMSEQ | B.PA_DEVERR_DECODE_QLEN)
            op.restore(t["kc"], t["vc"], t["scales"], t["cum"], t["past"], t["table"], 6)


@pytest.mark.parametrize("q,past,nd", [([1, 1, 1], [70, 3, 200], 3), ([5, 2], [40, 100], 0), ([70, 40], [30, 100], 0)])
def test_caches_beyond_4_gb(q, past, nd):
    """Pages at both ends of caches of 6 GB answer as those of a small one."""
    c = Case(q, past, kv=8, heads=16, hs=256, bs=64, seed=33)
    t, op = c.tensors(), c.op()
    want = c.forward(op, t, nd)
    small = c.p["num_blocks"]
    big = 6 * 2 ** 30 // (64 * 8 * 256)
    place = torch.arange(small, device="cuda") * ((big - 1) // (small - 1))
    place[-1] = big - 1
    c.p["num_blocks"] = big
    far, op = c.tensors(), c.op()
    for name in ("kc", "vc", "scales"):
        whole = torch.empty(big, *far[name].shape[1:], dtype=far[name].dtype, device="cuda")
        whole[place] = far[name]
        far[name] = whole
    far["table"] = torch.where(far["table"] >= 0, place[far["table"].long().clamp(min=0)].int(), -1).contiguous()
    far["slots"] = (place[far["slots"].long() // 64] * 64 + far["slots"].long() % 64).int()
    out = c.forward(op, far, nd)
    assert op.error_flags() == 0 and torch.equal(out, want)
    for name in ("kc", "vc", "scales"):
        assert torch.equal(far[name][place].view(torch.uint8), t[name].view(torch.uint8))
    rows = lambda op, t: op.restore(t["kc"], t["vc"], t["scales"], t["cum"], t["past"], t["table"], c.T)
    c.p["num_blocks"] = small
    for a, b in zip(rows(op, far), rows(c.op(), t)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("heads,kv", [(128, 1), (96, 1), (127, 1), (33, 3), (35, 5)])
@pytest.mark.parametrize("q", [1, 3, 40])
def test_large_and_odd_groups(heads, kv, q):
    _run(Case([q, q, 0], [70, 5, 30], heads=heads, kv=kv, hs=32, vhs=48, rd=16, seed=34), 2 if q == 1 else 0)


@pytest.mark.parametrize("kw", [dict(bs=4096, past=[5000, 0, 4095]), dict(bs=16, past=[0, 0, 0], hs=16, vhs=16, rd=16, heads=1, kv=1),
                                dict(bs=4096, past=[9000, 4096, 1], window=100)])
@pytest.mark.parametrize("q", [1, 70])
def test_page_sizes_at_the_ends(kw, q):
    _run(Case([q] * 3, seed=35, spare=0, **kw), 3 if q == 1 else 0)


def test_thousands_of_sequences():
    rng = np.random.default_rng(36)
    n = 2300
    _run(Case([1] * n, list(rng.integers(0, 60, n)), kv=1, heads=2, hs=16, seed=36), n)
    _run(Case(list(rng.integers(0, 3, n)), list(rng.integers(0, 60, n)), kv=1, heads=2, hs=16, seed=37), 0)
    n = 500
    _run(Case(list(rng.integers(0, 60, n)), list(rng.integers(0, 60, n)), kv=1, heads=2, hs=16, seed=38), 0)


def test_two_objects_at_once():
    """Objects on streams of their own, and graphs of one object replayed in turn."""
    cases = [Case([1] * 20 + [90, 300], list(range(100, 2100, 100)) + [800, 50], heads=8, kv=2, hs=128, bs=64, seed=s) for s in (40, 41)]
    want = [c.forward(c.op(), c.tensors(), 20).clone() for c in cases]
    ops, ts = [c.op() for c in cases], [c.tensors() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i in (0, 1):
            outs[i].append(cases[i].forward(ops[i], ts[i], 20, stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in (0, 1) for o in outs[i])
    graphs, held = [], [torch.zeros_like(w) for w in want]
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cases[i].forward(ops[0], ts[i], 20, out=held[i])
        graphs.append(g)
    for _ in range(5):
        for i in (0, 1):
            held[i].zero_()
            graphs[i].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(held[i], want[i]) for i in (0, 1))


def test_pages_in_two_tables():
    """A prefix that two sequences share, read by both."""
    c = Case([1, 1, 40, 40], [200, 230, 160, 170], seed=42)
    c.table[1, :12], c.table[3, :10] = c.table[0, :12], c.table[2, :10]
    for nd in (2, 0):
        t, op = c.tensors(), c.op()
        out = c.forward(op, t, nd)
        assert op.error_flags() == 0
        _check_out(out, *c.oracle([t["kc"].cpu().numpy(), t["vc"].cpu().numpy(), t["scales"].cpu().numpy()]))


@pytest.mark.parametrize("nd", [0, 2])
def test_rows_behind_the_last_sequence(nd):
    c = Case([1, 1], [20, 30], seed=20)
    t, op = c.tensors(), c.op()
    pad = lambda x: torch.cat([x, torch.zeros(3, x.size(1), dtype=x.dtype, device="cuda")])
    out = torch.full((5, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    c.forward(op, t, nd)
    op.attend(pad(t["query"]), t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["cum"], t["past"], t["table"], nd, out=out)
    assert bool((out[2:] == 7).all())
    ref, tol = c.oracle(c.oracle_write())
    _check_out(out[:2], ref, tol)


def test_arguments_refused():
    api = _api()
    PaError = _binding().PaError
    c = Case([2, 1], [20, 30], seed=21)
    t, op = c.tensors(), c.op()
    def bad(**over):
        with pytest.raises(PaError):
            c.forward(op, {**t, **over}, 0)
    bad(query=t["query"].float())
    bad(query=t["query"][:, :-1])
    bad(query=t["query"][:2].contiguous())
    bad(key=t["key"].half())
    bad(value=t["value"][:, ::2])
    bad(kc=t["kc"].int())
    bad(kc=t["kc"][:-1])
    bad(scales=t["scales"].double())
    bad(scales=t["scales"][:, :, :1].contiguous())
    bad(cum=t["cum"].long())
    bad(cum=t["cum"][:2].contiguous())
    bad(table=t["table"].cpu())
    bad(slots=t["slots"][:2].contiguous())
    bad(sink=torch.zeros(7, dtype=torch.bfloat16, device="cuda"))
    bad(q_norm=torch.zeros(7, dtype=torch.bfloat16, device="cuda"))
    bad(k_norm=torch.zeros(64, device="cuda"))
    bad(cos=t["cos"][:, :8].contiguous())
    with pytest.raises(PaError):
        c.forward(op, t, 3)
    with pytest.raises(PaError):
        op.restore(t["kc"], t["vc"], t["scales"], t["cum"], t["past"], t["table"][:1].contiguous(), 3)
    with pytest.raises(PaError):
        op.restore(t["kc"], t["vc"], t["scales"], t["cum"], t["past"], t["table"], 3, key=t["key"][:2])
    x = Case([2, 1], [20, 30], cross=1, seed=21)
    with pytest.raises(PaError):
        xt = x.tensors()
        x.op().forward(xt["query"], xt["key"], xt["value"], xt["kc"], xt["vc"], xt["scales"], None, None, xt["cum"], xt["past"],
                       xt["table"], xt["slots"], 0)
    with pytest.raises(PaError):
        api.QuantizedAttention(**dict(x.p, dtype=torch.float32), max_seqs=1, max_tokens=1)
    assert op.error_flags() == 0


@pytest.mark.parametrize("name", ["query", "key", "value", "kc", "vc", "scales", "cos", "sin", "cum", "past", "table", "slots"])
def test_a_tensor_left_out_is_refused_as_a_bad_argument(name):
    PaError = _binding().PaError
    c = Case([2, 1], [20, 30], seed=21)
    t, op = c.tensors(), c.op()
    with pytest.raises(PaError):
        c.forward(op, {**t, name: None}, 0)
    if name in ("query", "kc", "vc", "scales", "cos", "sin", "cum", "past", "table"):
        x = {**t, name: None}
        with pytest.raises(PaError):
            op.attend(x["query"], x["kc"], x["vc"], x["scales"], x["cos"], x["sin"], x["cum"], x["past"], x["table"], 0)
        out = torch.empty(3, 512, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(PaError):
            op.prefill(x["query"], x["kc"], x["vc"], x["scales"], x["cos"], x["sin"], x["cum"], x["past"], x["table"], out)
    if name in ("key", "value", "kc", "vc", "scales", "cos", "sin", "cum", "past", "slots"):
        x = {**t, name: None}
        with pytest.raises(PaError):
            op.write(x["key"], x["value"], x["kc"], x["vc"], x["scales"], x["cos"], x["sin"], x["slots"], x["cum"], x["past"])
    if name in ("kc", "vc", "scales", "cum", "past", "table"):
        x = {**t, name: None}
        with pytest.raises(PaError):
            op.restore(x["kc"], x["vc"], x["scales"], x["cum"], x["past"], x["table"], 3)
    with pytest.raises(PaError):
        op.decode(t["query"], t["kc"], t["vc"], t["scales"], t["cos"], t["sin"], t["cum"], t["past"], t["table"], None)
    assert op.error_flags() == 0


def test_nothing_to_do():
    c = Case([0, 0], [20, 30], seed=22)
    t, op = c.tensors(), c.op()
    assert c.forward(op, t, 0).shape == (0, 512)
    k, v = op.restore(t["kc"], t["vc"], t["scales"], t["cum"], t["past"], t["table"], 0)
    assert k.shape == (0, 128) and op.error_flags() == 0


# ------------------------------------------------------------------------- streams, graphs, repetition

def test_same_bits_every_time():
    for kw, nd in ((dict(q=[1] * 7, past=[10, 2000, 0, 900, 33, 64, 1500], heads=32, kv=2), 7),
                   (dict(q=[60, 7], past=[900, 2500], hs=128), 0)):
        c = Case(seed=23, **kw)
        t, op = c.tensors(), c.op()
        first = c.forward(op, t, nd).clone()
        codes = t["kc"].clone()
        for _ in range(5):
            assert torch.equal(c.forward(op, t, nd), first)
        assert torch.equal(t["kc"], codes)


def test_captured_and_replayed():
    c = Case([1, 1, 30], [200, 77, 100], sink=True, seed=24)
    t, op = c.tensors(), c.op()
    want = c.forward(op, t, 2).clone()
    out = torch.zeros_like(want)
    t2 = c.tensors()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.forward(op, t2, 2, out=out)
        k, v = op.restore(t2["kc"], t2["vc"], t2["scales"], t2["cum"], t2["past"], t2["table"], c.T)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert torch.equal(k, op.restore(t["kc"], t["vc"], t["scales"], t["cum"], t["past"], t["table"], c.T)[0])
    # other inputs in the same memory
    c2 = Case([1, 1, 30], [200, 77, 100], sink=True, seed=25)
    t3, fresh = c2.tensors(), c2.op()
    want = c2.forward(fresh, t3, 2)
    fill = c2.tensors()
    for name in t2:
        if t2[name] is not None:
            t2[name].copy_(fill[name])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_other_streams():
    c = Case([1, 1, 30], [200, 77, 100], seed=26)
    want = c.forward(c.op(), c.tensors(), 2).clone()
    for make in (lambda s: s, lambda s: s.cuda_stream):
        t, s = c.tensors(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        out = c.forward(c.op(), t, 2, stream=make(s))
        s.synchronize()
        assert torch.equal(out, want)


def test_float8_tensors():
    c = Case([1, 9], [30, 20], seed=27)
    t = c.tensors()
    want = c.forward(c.op(), c.tensors(), 0)
    t["kc"], t["vc"] = t["kc"].view(torch.float8_e4m3fn), t["vc"].view(torch.float8_e4m3fn)
    assert torch.equal(c.forward(c.op(), t, 0), want)


# -------------------------------------------------------------------------------- a run of them together

def test_serving_run_with_pages():
    """Prompts, steps, beams that fork in the middle of a page, a freed sequence and a compaction, with the
    scales carried by the pool; then the rows read back and attended by the 16-bit mode."""
    api = _api()
    dt, kv, heads, hs, bs, blocks, seqs, mb = torch.bfloat16, 3, 6, 64, 16, 40, 4, 8
    op = api.QuantizedAttention(dtype=dt, num_heads=heads, kv_num_heads=kv, head_size=hs, rotary_dim=hs, cos_rows=128,
                                block_size=bs, num_blocks=blocks, max_blocks_per_seq=mb, max_seqs=seqs, max_tokens=128,
                                own_slots=True)
    kc, vc, scales = op.new_caches()
    pool = api.PagePool([kc, vc], block_size=bs, max_seqs=seqs, max_blocks_per_seq=mb, page_tensors=[scales])
    p = dict(dtype=P.BF16, num_heads=heads, kv_num_heads=kv, head_size=hs, v_head_size=hs, rotary_offset=0, rotary_dim=hs,
             rotary_interleaved=0, cos_rows=128, block_size=bs, scale=0.0, softcap=0.0, local_window_size=-1, rms_eps=0.0, cross=0)
    ang = np.arange(128)[:, None] * 10000.0 ** (-np.arange(hs // 2)[None] / (hs // 2))
    cos, sin = P.round_f64(np.cos(ang), P.BF16), P.round_f64(np.sin(ang), P.BF16)
    dc, ds = (torch.from_numpy(x).to("cuda", dt) for x in (cos, sin))
    rng = np.random.default_rng(0)

    def step(lengths):
        T = sum(lengths)
        x = [P.round_f64(rng.standard_normal((T, n, hs)) * f, P.BF16) for n, f in ((heads, 1), (kv, rng.uniform(0.5, 4)), (kv, 1))]
        d = [torch.from_numpy(a).to("cuda", dt).view(T, -1) for a in x]
        cum = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
        dcum = torch.from_numpy(cum).cuda()
        slots = torch.empty(T, dtype=torch.int32, device="cuda")
        pool.reserve(dcum, slots)
        before = [a.cpu().numpy().copy() for a in (kc, vc, scales)]
        past, table = pool.past.cpu().numpy(), pool.block_table.cpu().numpy()
        out = op.forward(*d, kc, vc, scales, dc, ds, dcum, pool.past, pool.block_table, slots, 0)
        Q.write(x[1], x[2], cos, sin, slots.cpu().numpy(), cum, past, *before, p)
        assert (kc.cpu().numpy() == before[0]).all() and (scales.cpu().numpy() == before[2]).all()
        ref, tol = Q.attend(x[0], *before, cos, sin, cum, past, table, p)
        _check_out(out, ref, tol)
        pool.past += dcum[1:] - dcum[:-1]

    dev = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    step([37, 0, 20, 0])
    step([1, 0, 1, 0])
    pool.fork(dev(0, 2), dev(1, 3))
    for _ in range(3):
        step([1, 1, 1, 1])
    pool.free(dev(0))
    pool.compact()
    step([0, 2, 1, 5])
    step([50, 1, 1, 1])
    assert op.error_flags() == 0 and pool.error_flags() == 0

    # read back: a 16-bit cache of the same pages answers alike
    n = pool.past.cpu().numpy()
    T = int(n.sum())
    cum = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
    key, value = op.restore(kc, vc, scales, cum, torch.zeros_like(pool.past), pool.block_table, T)
    seq = np.repeat(np.arange(seqs), n)
    pos = np.arange(T) - np.concatenate([[0], np.cumsum(n)])[seq]
    rows = torch.from_numpy(pool.block_table.cpu().numpy()[seq, pos // bs].astype(np.int64) * bs + pos % bs).cuda()
    k16, v16 = (torch.zeros(blocks * bs, kv * hs, dtype=dt, device="cuda").index_copy_(0, rows, x) for x in (key, value))
    sep = api.SeparateAttention(dtype=dt, num_heads=heads, kv_num_heads=kv, head_size=hs, block_size=bs, num_blocks=blocks,
                                max_blocks_per_seq=mb, max_seqs=seqs, max_tokens=seqs)
    new = [torch.randn(seqs, m * hs, device="cuda").to(dt) for m in (heads, kv, kv)]
    one = torch.arange(seqs + 1, dtype=torch.int32, device="cuda")
    none = torch.full((seqs,), -1, dtype=torch.int32, device="cuda")
    last = pool.past - 1
    a = sep.forward(*new, k16, v16, None, None, one, last, pool.block_table, none, seqs)
    plain = api.QuantizedAttention(dtype=dt, num_heads=heads, kv_num_heads=kv, head_size=hs, block_size=bs,
                                   num_blocks=blocks, max_blocks_per_seq=mb, max_seqs=seqs, max_tokens=seqs)
    b = plain.attend(new[0], kc, vc, scales, None, None, one, last, pool.block_table, seqs)
    # both are within their roundings of the same numbers: those of bf16 operands (2^-8) and of bf16 results
    assert float((a.double() - b.double()).norm() / b.double().norm()) < 4 * 2.0 ** -8


def test_pool_copies_whole_page_tensors():
    """Scales of 8 bytes a page and more, beside caches of rows, by a few pairs and by many."""
    api = _api()
    for kv, n in ((1, 5), (3, 100), (300, 7)):
        rng = np.random.default_rng(kv)
        cache = torch.from_numpy(rng.integers(0, 256, (256, 16, 32)).astype(np.uint8)).cuda()
        scales = torch.from_numpy(rng.standard_normal((256, kv, 2)).astype(np.float32)).cuda()
        want, wc = scales.cpu().numpy().copy(), cache.cpu().numpy().copy()
        pool = api.PagePool([cache], block_size=16, max_seqs=2, max_blocks_per_seq=4, page_tensors=[scales])
        perm = rng.permutation(256)
        src, dst, rows = perm[:n], perm[n:2 * n], rng.integers(0, 17, n)
        for s, d, r in zip(src, dst, rows):
            wc[d, :r] = wc[s, :r]
            if r:
                want[d] = want[s]
        pool.copy(*(torch.from_numpy(x.astype(np.int32)).cuda() for x in (src, dst, rows)))
        assert pool.error_flags() == 0
        assert (cache.cpu().numpy() == wc).all() and (scales.cpu().numpy() == want).all()
    with pytest.raises(_binding().PaError):
        api.PagePool([cache], block_size=16, max_seqs=2, max_blocks_per_seq=4, page_tensors=[scales[:8]])
    with pytest.raises(_binding().PaError):
        api.PagePool([cache], block_size=16, max_seqs=2, max_blocks_per_seq=4, page_tensors=[scales[:, :, :1]])
