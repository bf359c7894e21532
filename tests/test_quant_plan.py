"""How reads over 8-bit caches are spread over the GPU (csrc/pa_quant_plan.h): plain host arithmetic, compiled
by itself."""
import ctypes
import itertools
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_latent_attention_cache_gb300", "csrc")
SHIM = r"""
#include "pa_quant_plan.h"
using namespace pa::quant;
extern "C" {
int64_t tokens_of(int64_t t, int64_t b, int64_t n) { return range_tokens(t, b, n); }
void choose(int64_t t, int64_t n, int64_t group, int* out) {
  const ReadChoice c = choose_kernels(t, n, group);
  out[0] = c.few; out[1] = c.rows; out[2] = c.many;
}
void grid_of(int64_t t, int64_t r, int64_t n, int64_t few, int64_t kvh, int64_t per, int64_t tiles, int sms,
             int64_t* out) {
  const PrefillGrid g = prefill_grid(t, r, n, few, kvh, per, tiles, sms);
  out[0] = g.ctas; out[1] = g.planned; out[2] = g.splits; out[3] = g.launched();
}
void write_of(int64_t t, int64_t n, int64_t kvh, int bs, int lanes, int row_bytes, int sms, int64_t* out) {
  const WritePlan w = write_plan(t, n, kvh, bs, lanes, row_bytes, sms);
  out[0] = w.threads; out[1] = w.cap; out[2] = w.runs;
}
void part_of(int cta, int planned, int splits, int* out) {
  const PrefillPart p = prefill_part(cta, planned, splits);
  out[0] = p.at; out[1] = p.split; out[2] = p.splits;
}
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SHIM)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(d / "plan.cpp"), "-o",
                    str(d / "plan.so")], check=True)
    lib = ctypes.CDLL(str(d / "plan.so"))
    i64 = ctypes.c_int64
    lib.tokens_of.restype, lib.tokens_of.argtypes = i64, [i64] * 3
    lib.choose.argtypes = [i64] * 3 + [ctypes.POINTER(ctypes.c_int)]
    lib.grid_of.argtypes = [i64] * 7 + [ctypes.c_int, ctypes.POINTER(i64)]
    lib.write_of.argtypes = [i64] * 3 + [ctypes.c_int] * 4 + [ctypes.POINTER(i64)]
    lib.part_of.argtypes = [ctypes.c_int] * 3 + [ctypes.POINTER(ctypes.c_int)]

    class Plan:
        tokens = staticmethod(lib.tokens_of)

        @staticmethod
        def grid(tokens, planned, nseq, *a, few=0):
            out = (i64 * 4)()
            lib.grid_of(tokens, planned, nseq, few, *a, out)
            return tuple(out)

        @staticmethod
        def choose(*a):
            out = (ctypes.c_int * 3)()
            lib.choose(*a, out)
            return out[0], bool(out[1]), bool(out[2])

        @staticmethod
        def write(*a):
            out = (i64 * 3)()
            lib.write_of(*a, out)
            return tuple(out)

        @staticmethod
        def part(*a):
            out = (ctypes.c_int * 3)()
            lib.part_of(*a, out)
            return tuple(out)
    return Plan


def test_a_range_beside_decode_sequences_is_planned_as_by_itself(plan):
    for decode, new, nseq in itertools.product((0, 1, 7, 200, 1000), (4, 20, 200, 4096), (1, 4)):
        tokens = plan.tokens(decode + new, decode + nseq, nseq)
        assert tokens == new == plan.tokens(new, nseq, nseq)
        alone = plan.grid(new, new, nseq, 8, 64, 100, 152)
        both = plan.grid(decode + new, tokens, nseq, 8, 64, 100, 152)
        assert both[1:3] == alone[1:3] and alone[0] == alone[1]


def test_whatever_the_offsets_every_unit_has_its_place(plan):
    """Sequences outside the range without tokens, ranges in the middle, one token, many sequences."""
    for num_tokens, num_seqs, nseq, kvh, per, tiles, sms in itertools.product(
            (1, 5, 300, 4000), (1, 3, 256, 4096), (1, 2, 200), (1, 8), (1, 64, 256), (1, 9, 1000), (1, 148, 152)):
        if nseq > num_seqs:
            continue
        tokens = plan.tokens(num_tokens, num_seqs, nseq)
        assert 1 <= tokens <= num_tokens
        ctas, planned, splits, launched = plan.grid(num_tokens, tokens, nseq, kvh, per, tiles, sms)
        assert 1 <= planned <= ctas and splits >= 1 and launched == ctas + planned * (splits - 1)
        # units of any offsets that rise: all in one sequence, or spread over as many as there are
        for n in (1, min(nseq, num_tokens)):
            assert ((num_tokens - n + 1 + per - 1) // per + n - 1) * kvh <= ctas
        assert splits == 1 or planned * splits <= sms  # (the workspace holds as many parts)
        assert splits == 1 or splits <= tiles // 4


def test_parts_cover_every_unit_once(plan):
    for planned, splits, more in itertools.product((1, 3, 16), (1, 2, 9), (0, 1, 40)):
        seen = {}
        for cta in range(planned * splits + more):
            at, split, n = plan.part(cta, planned, splits)
            assert 0 <= split < n
            if n > 1:
                assert cta == at * n + split < planned * splits  # (where the joining kernel looks for it)
            assert seen.setdefault(at, n) == n or split == 0
            seen[(at, split)] = cta
        units = sorted(k for k in seen if isinstance(k, int))
        assert units == list(range(planned + more))
        assert all((at, s) in seen for at in units for s in range(seen[at]))
        assert sum(isinstance(k, tuple) for k in seen) == planned * splits + more


def test_write_holds_what_its_runs_bring(plan):
    """In pieces of whole rounds of its threads, within its shared memory; single tokens of large batches do
    not each hold room for a page."""
    for tokens, seqs, kvh, bs, (hs, vhs) in itertools.product(
            (1, 32, 200, 5000, 100000), (1, 32, 512, 5000), (1, 8), (16, 64, 128, 4096),
            ((16, 16), (64, 128), (128, 128), (192, 128), (256, 256), (16, 256))):
        lanes = 2
        while lanes * 8 < max(hs, vhs):
            lanes *= 2
        row = (2 * hs + vhs) * 2
        threads, cap, runs = plan.write(tokens, seqs, kvh, bs, lanes, row, 152)
        assert threads in (128, 256, 512) and cap > 0 and cap % (threads // lanes) == 0
        assert cap * row <= (96 if threads == 512 else 48) * 1024 and cap < bs + threads // lanes
        assert runs >= 2 * seqs + tokens // bs
        waves = runs * kvh / (152 * (228 * 1024 // (cap * row + bs + 1024)))
        brings = max(8, min(bs, -(-tokens // seqs)))
        assert waves <= 1 or cap < brings + threads // lanes
    assert plan.write(512, 512, 8, 64, 16, 768, 152)[:2] == (128, 8)
    assert plan.write(32, 32, 8, 64, 16, 768, 152)[:2] == (128, 64)
    assert plan.write(14740, 4, 8, 64, 16, 768, 152)[:2] == (256, 64)


def test_a_long_sequence_among_short_ones_has_the_kernel_for_long_ones(plan):
    """Both kernels where a batch of few rows on average may hold a long sequence, and no row without a kernel."""
    for tokens, nseq, group in itertools.product((1, 4, 80, 640, 3300, 100000), (1, 2, 16, 301, 5000), (1, 3, 4, 16, 128)):
        few, rows, many = plan.choose(tokens, nseq, group)
        assert rows or many
        assert rows == (tokens * group <= 48 * nseq) and (few > 0) == rows
        if not many:  # whatever the offsets, no sequence is long
            assert tokens * group <= 2048 and few >= tokens
        if rows and many:
            assert 48 < few * group <= 1024 and (few + 1) * group > 1024 and few < tokens
    assert plan.choose(3300, 301, 4) == (256, True, True)
    assert plan.choose(80, 16, 4)[1:] == (True, False)
    assert plan.choose(2000, 1, 4) == (0, False, True)


def test_long_sequences_have_a_place_each(plan):
    """Beside any number of short ones, as many long ones as the tokens allow."""
    for tokens, nseq, per, few in itertools.product((700, 3300, 100000), (15, 301, 5000), (1, 64, 256), (8, 256, 1024)):
        if tokens <= few:
            continue
        ctas, planned, splits, launched = plan.grid(tokens, tokens, nseq, 8, per, 1000, 152, few=few)
        assert 1 <= planned <= ctas and launched == ctas + planned * (splits - 1)
        assert splits == 1 or planned * splits <= 152
        for n in {1, 2, min(nseq, tokens // (few + 1))}:  # n long ones, all but one just long enough
            last = tokens - (n - 1) * (few + 1)
            if n >= 1 and last > few:
                assert (-(-last // per) + (n - 1) * -(-(few + 1) // per)) * 8 <= ctas
