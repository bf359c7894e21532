"""Differential attention on the GPU against the oracle.

Tolerances: cache rows within 1 ulp where RoPE touches them and bit-equal
elsewhere. Outputs: |err| <= 6 u noise, u the largest relative rounding error
of the dtype (2^-8 bf16, 2^-11 fp16) and ``noise`` the oracle's sum of how far
a rounding of size 1 of the probabilities, the query operand and the output
moves an output: independent roundings of at most u have a standard deviation
of u / sqrt(3) times that, so 6 u is over ten of them. On top 2^-20 of the
largest output of the head for the f32 arithmetic (ex2, sums, norm)."""
import numpy as np
import pytest
import torch

from oracle import diff_oracle as D
from paged_latent_attention_cache_gb300 import binding as B
from paged_latent_attention_cache_gb300 import workloads as W
from paged_latent_attention_cache_gb300.api import DifferentialAttention, PagePool
from tests.harness import UNIT_ROUNDOFF, _ordered

pytestmark = pytest.mark.gpu


def _numpy(w):
    return {k: W.to_bits(v) if v.dtype in (torch.bfloat16, torch.float16) else v.numpy()
            for k, v in w.tensors.items()}


def _op(w, **kw):
    return DifferentialAttention(**w.params, max_seqs=max(len(w.q_lens), 1),
                                 max_tokens=max(w.num_tokens, 1), **{"own_slots": True, **kw})


def _args(d):
    return (d["query"], d["key"], d["value"], d["key_cache"], d["value_cache"], d["cos_cache"],
            d["sin_cache"], d["lambda_vectors"], d["norm_weight"], d["cumseq"], d["past"],
            d["block_table"], d["slot_mapping"])


def run_gpu(w, decodes=None, op=None):
    d = {k: v.cuda() for k, v in w.tensors.items()}
    op = op or _op(w)
    out = torch.full((w.num_tokens, w.num_heads * w.v_head_size), float("nan"), dtype=w.dtype,
                     device="cuda")
    op.forward(*_args(d), w.num_decode_seqs if decodes is None else decodes, out=out)
    torch.cuda.synchronize()
    return d, out, op


def check(w, tokens=None, decodes=None):
    d, out, op = run_gpu(w, decodes)
    assert op.error_flags() == 0, hex(op.error_flags())
    tag = W.dtype_tag(w.dtype)
    ref = D.run_bits(_numpy(w), w.params, tag, tokens)
    assert np.array_equal(W.to_bits(d["value_cache"]), ref["value_cache"])
    k0, k1 = W.to_bits(d["key_cache"]), ref["key_cache"]
    ulp = np.abs(_ordered(k0) - _ordered(k1))
    rot = np.zeros(w.head_size, bool)
    rot[w.rotary_offset:w.rotary_offset + w.rotary_dim] = True
    assert ulp[..., ~rot].max(initial=0) == 0 and ulp.max() <= 1
    o = out if tokens is None else out[torch.as_tensor(list(tokens))]
    got = o.double().cpu().numpy().reshape(ref["out"].shape)
    assert np.isfinite(got).all()
    err = np.abs(got - ref["out"])
    bound = 6 * UNIT_ROUNDOFF[w.dtype] * ref["noise"] + 2.0 ** -20 * np.abs(ref["out"]).max(-1, keepdims=True)
    worst = (err / bound).max()
    rel = np.linalg.norm(got - ref["out"]) / np.linalg.norm(ref["out"])
    print(f"RATIO {w.name}: {worst:.3f} of the bound, relative error {rel:.2e}")
    assert worst <= 1, worst


BASE = dict(q_lens=[1, 1, 1, 9, 0, 40, 130], past_lens=[700, 0, 63, 70, 5, 3, 129], num_heads=8,
            kv_num_heads=2, head_size=64, block_size=64, seed=11, drop_slots=2)

VARIANTS = {
    "64_128": {},
    "128_256": dict(head_size=128),
    "fp16": dict(dtype=torch.float16),
    "fp16_128_256": dict(dtype=torch.float16, head_size=128, num_heads=4),
    "mha": dict(num_heads=4, kv_num_heads=4),
    "mqa_16": dict(num_heads=16, kv_num_heads=1),
    "grp_3": dict(num_heads=6, kv_num_heads=2),
    "grp_12": dict(num_heads=12, kv_num_heads=1, head_size=32),
    "grp_40": dict(num_heads=40, kv_num_heads=1, head_size=32),
    "grp_128": dict(num_heads=128, kv_num_heads=1, head_size=16, q_lens=[1, 5], past_lens=[90, 40]),
    "hs_16": dict(head_size=16),
    "hs_48_vhs_80": dict(head_size=48, v_head_size=80),
    "hs_96_vhs_192": dict(head_size=96),
    "vhs_8": dict(v_head_size=8),
    "vhs_136": dict(v_head_size=136),
    "vhs_64": dict(v_head_size=64),
    "hs_128_vhs_64": dict(head_size=128, v_head_size=64),
    "bs_16": dict(block_size=16),
    "bs_128": dict(block_size=128),
    "bs_256": dict(block_size=256),
    "window_1": dict(local_window_size=0),
    "window_7": dict(local_window_size=7),
    "window_100": dict(local_window_size=100),
    "softcap": dict(softcap=2.0),
    "softcap_window": dict(softcap=5.0, local_window_size=33, dtype=torch.float16),
    "interleaved": dict(rotary_interleaved=1),
    "partial_rope": dict(rotary_dim=32, rotary_offset=16),
    "no_rope": dict(rotary_dim=0),
    "lambda_0.8": dict(lambda_init=0.8),
    "peaked": dict(std=4.0),
    "flat": dict(std=0.1, lambda_init=0.2),
    "scale": dict(scale=0.5),
}


def workload(name, **over):
    kw = {**BASE, **VARIANTS[name], **over}
    return W.make_diff_workload(name, kw.pop("q_lens"), kw.pop("past_lens"), **kw)


@pytest.mark.parametrize("name", sorted(VARIANTS))
def test_variants(name):
    check(workload(name))


@pytest.mark.parametrize("name", ["64_128", "128_256", "window_7"])
def test_decodes_as_prefill(name):
    """One-token sequences through the prefill call."""
    check(workload(name, q_lens=[1, 1, 1], past_lens=[700, 0, 63]), decodes=0)


@pytest.mark.parametrize("past", [0, 1, 14, 15, 16, 31, 62, 63, 64, 65, 126, 127, 128, 129, 255, 256, 511, 1023])
def test_decode_lengths(past):
    """Context lengths around every tile and page boundary."""
    check(workload("64_128", q_lens=[1], past_lens=[past], block_size=16, num_heads=2, drop_slots=0))


@pytest.mark.parametrize("q,past", [(2, 0), (31, 0), (32, 1), (33, 95), (64, 64), (127, 1), (128, 0), (129, 127), (300, 20)])
def test_prefill_lengths(q, past):
    check(workload("64_128", q_lens=[q], past_lens=[past], block_size=16, num_heads=2, drop_slots=0))


@pytest.mark.parametrize("name,past", [
    ("64_128", [9000, 17, 300]), ("128_256", [9000, 17, 300]), ("128_256", [40000]), ("hs_96_vhs_192", [30000, 5]),
    ("hs_128_vhs_64", [30000, 5]), ("vhs_136", [30000, 5])])
def test_long_split_decode(name, past):
    """Long sequences, split over many CTAs whose rings turn many times, and joined."""
    check(workload(name, q_lens=[1] * len(past), past_lens=past, num_heads=4, drop_slots=0))


def test_many_sequences():
    rng = np.random.default_rng(0)
    check(workload("64_128", q_lens=[1] * 90, past_lens=[int(x) for x in rng.integers(0, 400, 90)], num_heads=2,
                   kv_num_heads=1, block_size=16))


@pytest.mark.parametrize("kind", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("name", ["64_128", "window_7", "128_256"])
def test_unseen_rows_may_hold_anything(kind, name):
    """Rows after a sequence's end in its last page, rows before its window
    and pages of nobody hold NaN or infinities: no output changes."""
    w = workload(name, block_size=128, num_blocks=16, drop_slots=0)
    _, want, _ = run_gpu(w)
    t = w.tensors
    seen = torch.zeros(t["key_cache"].shape[0] * 128, dtype=torch.bool)
    for b, (q, p) in enumerate(zip(w.q_lens, w.past_lens)):
        lo = max(0, p - w.local_window_size) if w.local_window_size >= 0 else 0
        if q:
            j = torch.arange(lo, p + q)
            seen[(t["block_table"][b, j // 128] * 128 + j % 128).long()] = True
    for k in ("key_cache", "value_cache"):
        t[k].view(len(seen), -1)[~seen] = kind
    _, got, op = run_gpu(w)
    assert op.error_flags() == 0
    assert torch.equal(got, want)


def test_flags_and_range_calls():
    """write + one read call per sequence range, with and without the
    after-write flags: bit-equal rows, other rows untouched."""
    w = workload("64_128", drop_slots=0)
    d, want, op = run_gpu(w)
    for after in (False, True):
        out = torch.full_like(want, -7.0)
        read = (d["query"], d["key_cache"], d["value_cache"], d["cos_cache"], d["sin_cache"],
                d["lambda_vectors"], d["norm_weight"], d["cumseq"], d["past"], d["block_table"], out)
        op.write(d["key"], d["value"], d["key_cache"], d["value_cache"], d["cos_cache"],
                 d["sin_cache"], d["slot_mapping"], d["cumseq"], d["past"])
        op.decode(*read, 0, 3, after_write=after)
        assert torch.equal(out[:3], want[:3]) and (out[3:] == -7).all()
        op.prefill(*read, 5, 6)
        assert torch.equal(out[12:52], want[12:52]) and (out[3:12] == -7).all() and (out[52:] == -7).all()
    assert op.error_flags() == 0


def test_graph_replay_two_graphs_one_workspace():
    """A decode step and a prefill step captured apart share one operator's
    workspace; replayed in turn they repeat the eager results bit for bit."""
    wd = workload("64_128", q_lens=[1] * 4, past_lens=[2000, 100, 0, 5], drop_slots=0)
    wp = workload("64_128", q_lens=[70, 3], past_lens=[100, 5], drop_slots=0, num_blocks=wd.num_blocks,
                  max_blocks_per_seq=wd.max_blocks_per_seq, cos_rows=wd.cos_rows)
    op = DifferentialAttention(**wd.params, max_seqs=4, max_tokens=128)
    dd, want_d, _ = run_gpu(wd, op=op)
    dp, want_p, _ = run_gpu(wp, op=op)
    outs, graphs = [], []
    for d, want, n in ((dd, want_d, 4), (dp, want_p, 0)):
        out = torch.zeros_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            op.forward(*_args(d), n, out=out)
        outs.append(out)
        graphs.append(g)
    side = torch.cuda.Stream()
    for k in (0, 1, 1, 0, 0):
        outs[k].fill_(3.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[k].replay()
        side.synchronize()
        assert torch.equal(outs[k], (want_d, want_p)[k])


@pytest.mark.parametrize("what", ["block", "context", "past", "position", "qlen", "slot"])
def test_bad_indices(what):
    """Bad pages, lengths, positions and slots set their flag; the rows of
    that sequence become zeros (or stay, for a wrong q_len), the others do not
    change: within one step of the dtype, 2 u |x|, as a decode is cut by the
    lengths of the whole batch and so sums in another order, where the f32 sums
    themselves differ by under 2^-20 of the largest output."""
    w = workload("64_128", q_lens=[1, 1, 20, 30], past_lens=[100, 200, 10, 50], drop_slots=0)
    _, want, _ = run_gpu(w)
    t = w.tensors
    if what == "block":
        t["block_table"][1, 2] = 10 ** 6
        t["block_table"][3, 0] = -1
        flag, zero = B.PA_DEVERR_BLOCK, [1, 3]
    elif what == "context":
        t["past"][1] = 10 ** 6
        t["past"][3] = w.max_blocks_per_seq * 64 - 10
        flag, zero = B.PA_DEVERR_CONTEXT, [1, 3]
    elif what == "past":
        t["past"][1], t["past"][3] = -5, -40
        flag, zero = B.PA_DEVERR_CONTEXT, [1, 3]
    elif what == "position":
        w.params["cos_rows"] = 150
        flag, zero = B.PA_DEVERR_POSITION, [1]
    elif what == "qlen":
        flag, zero = B.PA_DEVERR_DECODE_QLEN, []
    else:
        t["slot_mapping"][0], t["slot_mapping"][5] = 10 ** 8, -2
        flag, zero = B.PA_DEVERR_SLOT, []
    op = _op(w, own_slots=False)
    _, got, _ = run_gpu(w, op=op, decodes=3 if what == "qlen" else None)
    assert op.error_flags() & flag, hex(op.error_flags())
    assert op.error_flags() & ~(flag | B.PA_DEVERR_CONTEXT | B.PA_DEVERR_POSITION) == 0
    cum = t["cumseq"].tolist()
    for b in range(4):
        rows = got[cum[b]:cum[b + 1]]
        if b in zero:
            assert (rows == 0).all() or (what in ("context", "past") and b == 3), b
            if b == 3:
                assert torch.isfinite(rows.float()).all()
        elif what == "qlen" and b == 2:
            assert torch.isnan(rows.float()).all()
        elif what != "slot":
            x, y = rows.double(), want[cum[b]:cum[b + 1]].double()
            step = 2 * UNIT_ROUNDOFF[w.dtype] * torch.maximum(x.abs(), y.abs())
            assert ((x - y).abs() <= step + 2.0 ** -20 * y.abs().max()).all(), b


def test_rows_behind_the_last_sequence_stay():
    w = workload("64_128", q_lens=[1, 1, 20], past_lens=[100, 200, 10], drop_slots=0)
    d = {k: v.cuda() for k, v in w.tensors.items()}
    for k in ("query", "key", "value"):
        d[k] = torch.cat([d[k], d[k][:9]])
    d["slot_mapping"] = torch.cat([d["slot_mapping"], torch.full((9,), -1, dtype=torch.int32, device="cuda")])
    op = DifferentialAttention(**w.params, max_seqs=3, max_tokens=64)
    out = torch.full((31, w.num_heads * w.v_head_size), -7.0, dtype=w.dtype, device="cuda")
    op.forward(*_args(d), 2, out=out)
    _, want, _ = run_gpu(w)
    assert torch.equal(out[:22], want) and (out[22:] == -7).all()


def test_refuses_bad_tensors():
    w = workload("64_128", q_lens=[1, 4], past_lens=[10, 3], drop_slots=0)
    d, _, op = run_gpu(w)
    for name, bad in [("query", d["query"].float()), ("key", d["key"][:, ::2]), ("value", d["value"].cpu()),
                      ("cumseq", d["cumseq"].long()), ("past", d["past"][:1]), ("block_table", d["block_table"][:1]),
                      ("lambda_vectors", d["lambda_vectors"].double()), ("norm_weight", d["norm_weight"][:64]),
                      ("key_cache", d["key_cache"][:1]), ("cos_cache", d["cos_cache"][:2]),
                      ("slot_mapping", d["slot_mapping"][:2])]:
        e = dict(d)
        e[name] = bad
        with pytest.raises(B.PaError):
            op.forward(*_args(e), 1)


def test_serving_run_with_pages():
    """Prompts, forks, tokens and a compaction through a PagePool over both
    caches: forks answer as their parent, compaction changes no output bit."""
    w = workload("64_128", q_lens=[37, 64, 5, 0, 0], past_lens=[0] * 5, block_size=16, num_blocks=64,
                 max_blocks_per_seq=8, cos_rows=128, drop_slots=0)
    d = {k: v.cuda() for k, v in w.tensors.items()}
    pool = PagePool([d["key_cache"], d["value_cache"]], block_size=16, max_seqs=5, max_blocks_per_seq=8)
    op = _op(w)
    i32 = lambda v: torch.tensor(list(v), dtype=torch.int32, device="cuda")

    def step(q_lens, q, k, v, decodes):
        cum = i32([0] + list(np.cumsum(q_lens)))
        slots = pool.reserve(cum, torch.empty(sum(q_lens), dtype=torch.int32, device="cuda"))
        out = op.forward(q, k, v, d["key_cache"], d["value_cache"], d["cos_cache"], d["sin_cache"],
                         d["lambda_vectors"], d["norm_weight"], cum, pool.past, pool.block_table,
                         slots, decodes)
        pool.past += cum[1:] - cum[:-1]
        return out

    first = step(w.q_lens, d["query"], d["key"], d["value"], 0)
    _, want, _ = run_gpu(w)
    assert torch.equal(first, want)  # the same batch on other pages
    pool.free(i32([1]))
    pool.fork(i32([0, 0, 2]), i32([1, 3, 4]))
    pick = [0, 0, 1, 0, 1]
    out = step([1] * 5, d["query"][pick].contiguous(), d["key"][pick].contiguous(),
               d["value"][pick].contiguous(), 5)
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[3]) and torch.equal(out[2], out[4])

    def read():
        o = torch.zeros_like(out)
        op.decode(d["query"][pick].contiguous(), d["key_cache"], d["value_cache"], d["cos_cache"],
                  d["sin_cache"], d["lambda_vectors"], d["norm_weight"], i32(range(6)),
                  pool.past - 1, pool.block_table, o)
        return o

    before = read()
    assert torch.equal(before, out)
    pool.free(i32([0, 2]))
    pool.compact()
    after = read()
    assert torch.equal(before[[1, 3, 4]], after[[1, 3, 4]])
    assert pool.error_flags() == 0


def test_many_prompts():
    """More than 32 sequences with any number of new tokens, none among them."""
    rng = np.random.default_rng(1)
    q = [int(x) for x in rng.integers(0, 30, 45)]
    past = [int(x) for x in rng.integers(0, 200, 45)]
    w = workload("64_128", q_lens=q, past_lens=past, num_heads=2, kv_num_heads=1, block_size=16)
    check(w, decodes=0)


@pytest.mark.parametrize("name", ["64_128", "128_256"])
def test_maximum_moves_in_every_tile(name):
    """Keys that grow with their position: every tile's largest score passes
    the running maximum by far, so that O is scaled again and again."""
    w = workload(name, q_lens=[1, 200], past_lens=[1500, 900], drop_slots=0, rotary_dim=0, num_heads=4)
    t = w.tensors
    q = t["query"].view(w.num_tokens, 4, 2, -1)
    q.copy_(q.abs())
    for b, (n, p) in enumerate(zip(w.q_lens, w.past_lens)):
        j = torch.arange(p + n)
        rows = (t["block_table"][b, j // 64] * 64 + j % 64).long()
        kc = t["key_cache"].view(-1, 2, 2, w.head_size)
        grow = (j.float() / 25).view(-1, 1, 1, 1) * torch.tensor([1.0, 0.5]).view(1, 1, 2, 1)
        kc[rows] = (kc[rows].float() * 0.1 + grow).to(w.dtype)
    check(w)


def test_far_pages():
    """Pages beyond 2^32 bytes of both caches (and 2^31 elements of the keys)."""
    nb, bs, kv, hs = 70000, 64, 4, 64
    free = torch.cuda.mem_get_info()[0]
    if free < 40 << 30:
        pytest.skip("needs 20 GB of device memory")
    w = workload("64_128", q_lens=[1, 40], past_lens=[500, 100], kv_num_heads=kv, num_heads=8, drop_slots=0)
    d, want, _ = run_gpu(w)
    small = w.tensors["block_table"]
    t = {k: v.cuda() for k, v in w.tensors.items()}
    for k, width in (("key_cache", 2 * hs), ("value_cache", 128)):
        big = torch.full((nb, bs, kv, width), float("nan"), dtype=w.dtype, device="cuda")
        n = t[k].shape[0]
        big[nb - n:] = t[k].view(n, bs, kv, width)
        t[k] = big.view(nb, bs, kv, 2, hs) if k == "key_cache" else big
    n = w.num_blocks
    t["block_table"] = torch.where(small >= 0, small + nb - n, small).cuda()
    t["slot_mapping"] = torch.where(t["slot_mapping"] >= 0, t["slot_mapping"] + (nb - n) * bs, -1).int()
    op = DifferentialAttention(**{**w.params, "num_blocks": nb}, max_seqs=2, max_tokens=64)
    out = op.forward(*_args(t), 1)
    assert op.error_flags() == 0 and torch.equal(out, want)
    pool = PagePool([t["key_cache"], t["value_cache"]], block_size=bs, max_seqs=2, max_blocks_per_seq=4)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    pool.copy(i32(nb - 1, nb - 2), i32(1, nb - n - 1))
    for c in (t["key_cache"], t["value_cache"]):
        assert torch.equal(c[1].view(torch.int16), c[nb - 1].view(torch.int16))
        assert torch.equal(c[nb - n - 1].view(torch.int16), c[nb - 2].view(torch.int16))
    assert pool.error_flags() == 0


def test_two_operators_on_two_streams():
    """Two operators with workspaces of their own run at the same time, each on
    the stream it is given while another one is current."""
    wa = workload("64_128", q_lens=[1] * 6, past_lens=[3000, 10, 700, 64, 5, 900], drop_slots=0)
    wb = workload("128_256", q_lens=[1, 1, 90], past_lens=[2000, 17, 300], drop_slots=0)
    (da, want_a, _), (db, want_b, _) = run_gpu(wa), run_gpu(wb)
    oa, ob = _op(wa), _op(wb)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        outs.append((oa.forward(*_args(da), 6, stream=sa), ob.forward(*_args(db), 2, stream=sb)))
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, want_a) and torch.equal(b, want_b)


def test_nothing_to_do():
    w = workload("64_128", q_lens=[0, 0], past_lens=[10, 0], drop_slots=0)
    d, out, op = run_gpu(w)
    assert out.shape == (0, 8 * 128) and op.error_flags() == 0
    before = d["key_cache"].clone()
    op.forward(*_args(d), 0)
    torch.cuda.synchronize()
    assert torch.equal(before, d["key_cache"])


@pytest.mark.parametrize("name", ["64_128", "128_256"])
def test_same_bits_every_time(name):
    w = workload(name, q_lens=[1] * 20 + [150, 33], past_lens=list(range(0, 4000, 200)) + [1000, 5], drop_slots=0)
    op = _op(w)
    _, want, _ = run_gpu(w, op=op)
    for _ in range(10):
        _, got, _ = run_gpu(w, op=op)
        assert torch.equal(got, want)


def test_workspace_refused_before_launch():
    w = workload("64_128", q_lens=[1] * 3, past_lens=[3000, 10, 700], drop_slots=0)
    d, want, op = run_gpu(w)
    op.workspace = op.workspace[:256]
    with pytest.raises(B.PaError, match="workspace"):
        op.forward(*_args(d), 3)
    op.workspace = None
    with pytest.raises(B.PaError, match="workspace"):
        op.forward(*_args(d), 3)


def _row(w, b, j):
    """The cache row of position j of sequence b."""
    return int(w.tensors["block_table"][b, j // w.block_size]) * w.block_size + j % w.block_size


@pytest.mark.parametrize("name", ["64_128", "128_256", "mqa_16"])
def test_decode_nan_in_a_seen_key(name):
    """NaN in one seen key of one kv head and map: the rows of that head's
    queries are NaN, wherever in a long sequence and its parts the key lies;
    other heads and sequences do not change."""
    for at in (0, 17, 2500, 5000):
        w = workload(name, q_lens=[1, 1], past_lens=[5000, 100], drop_slots=0)
        _, want, _ = run_gpu(w)
        t = w.tensors
        kv, last = w.kv_num_heads, w.kv_num_heads - 1
        if at == 5000:  # the new token's own key
            t["key"].view(2, kv, 2, -1)[0, last, 1] = float("nan")
        else:
            t["key_cache"].view(-1, kv, 2, w.head_size)[_row(w, 0, at), last, 1] = float("nan")
        _, got, op = run_gpu(w)
        assert op.error_flags() == 0
        grp = w.num_heads // kv
        got, want = got.view(2, w.num_heads, -1), want.view(2, w.num_heads, -1)
        assert torch.isnan(got[0, last * grp:].float()).all()
        assert torch.equal(got[0, :last * grp], want[0, :last * grp]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("kind", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("name", ["64_128", "128_256", "fp16", "fp16_128_256", "window_7", "window_100", "grp_40", "vhs_136"])
def test_prefill_values_seen_by_some_rows(kind, name):
    """A value that is not finite reaches no token that does not see its key
    (an earlier one, or one whose window lies behind it): those rows are bit
    for bit what they are with zeros there. With NaN the others are NaN."""
    q, past = 90, 60
    w = workload(name, q_lens=[q], past_lens=[past], block_size=16, drop_slots=0)
    t = w.tensors
    kv, win = w.kv_num_heads, w.local_window_size
    rng = np.random.default_rng(3)
    for j in (past, past + 1, past + 37, past + 67, past + q - 1, past - 5):
        new = j >= past
        target = t["value"].view(q, kv, -1)[j - past] if new else \
            t["value_cache"].view(-1, kv, w.v_head_size)[_row(w, 0, j)]
        keep, c = target.clone(), int(rng.integers(0, w.v_head_size))
        outs = []
        for v in (0.0, kind):
            target[kv - 1, c] = v
            _, o, op = run_gpu(w, decodes=0)
            assert op.error_flags() == 0
            outs.append(o.view(q, kv, -1))
        target.copy_(keep)
        pos = torch.arange(past, past + q)
        sees = ((pos >= j) & ((pos - j <= win) if win >= 0 else (pos >= 0))).cuda()
        zero, got = outs
        assert torch.equal(got[:, :kv - 1], zero[:, :kv - 1])
        if kind != kind:
            assert torch.isnan(got[sees, kv - 1].float()).all()
        assert torch.equal(got[~sees, kv - 1], zero[~sees, kv - 1]), j


def test_more_sequences_than_tokens():
    """Empty sequences between a few tokens."""
    q = [0] * 200
    for b in (0, 63, 64, 150, 199):
        q[b] = 3
    past = [b % 40 for b in range(200)]
    check(workload("64_128", q_lens=q, past_lens=past, num_heads=2, kv_num_heads=1, block_size=16, drop_slots=0),
          decodes=0)


@pytest.mark.parametrize("name", ["64_128", "128_256"])
@pytest.mark.parametrize("window", [0, 31, 63, 64, 65, 100, 127, 128, 129, 200])
def test_prefill_windows(name, window):
    """Windows that begin anywhere in a tile of keys or in the half tiles that
    its values come in, or leave such a half to nobody."""
    check(workload(name, q_lens=[70, 150], past_lens=[301, 77], local_window_size=window, num_heads=4,
                   block_size=16, drop_slots=0))


@pytest.mark.parametrize("decodes", [0, None])
@pytest.mark.parametrize("name", ["64_128", "128_256", "fp16", "fp16_128_256", "hs_48_vhs_80", "grp_12", "window_100",
                                  "interleaved", "partial_rope", "no_rope", "lambda_0.8", "peaked"])
def test_as_exact_as_its_rounding(name, decodes):
    """The query and the probabilities enter the products as two parts, so they
    are off by u^2 at most (the remainder's rounding), and every output by its own
    rounding, u |x|, plus c noise: c = 6 u^2 for the parts (as 6 u above), and
    2^-15 for the f32 arithmetic: 6 deviations of sums of up to 1200 terms, 6 *
    sqrt(1200) * 2^-24 < 2^-16, and as much again for scores and exponentials."""
    w = workload(name)
    d, out, op = run_gpu(w, decodes)
    ref = D.run_bits(_numpy(w), w.params, W.dtype_tag(w.dtype))
    got = out.double().cpu().numpy().reshape(ref["out"].shape)
    u = UNIT_ROUNDOFF[w.dtype]
    bound = u * np.abs(ref["out"]) + (6 * u * u + 2.0 ** -15) * ref["noise"]
    worst = (np.abs(got - ref["out"]) / bound).max()
    print(f"RATIO {name}: {worst:.3f}")
    assert worst <= 1, worst


@pytest.mark.parametrize("name,offset,dim", [("64_128", 8, 32), ("64_128", 8, 16), ("64_128", 40, 16), ("128_256", 24, 80),
                                             ("128_256", 8, 112), ("128_256", 0, 0), ("hs_48_vhs_80", 8, 32),
                                             ("hs_16", 0, 16), ("fp16_128_256", 56, 64)])
@pytest.mark.parametrize("interleaved", [0, 1])
def test_rotations_that_end_in_a_k_step(name, offset, dim, interleaved):
    """Rotary ranges that start or end inside the 16 channels of a product."""
    check(workload(name, rotary_offset=offset, rotary_dim=dim, rotary_interleaved=interleaved))
    check(workload(name, rotary_offset=offset, rotary_dim=dim, rotary_interleaved=interleaved, q_lens=[1, 1, 30],
                   past_lens=[90, 3, 200]), decodes=0)


@pytest.mark.parametrize("gap", [14, 18, 22])
@pytest.mark.parametrize("name,q,past,at", [
    ("fp16", [1, 1], [32000, 700], 0), ("fp16", [1, 1], [32000, 700], 20000), ("fp16_128_256", [1], [9000], 5),
    ("fp16", [9, 3], [8000, 300], 0), ("fp16", [9], [8000], 6000), ("fp16_128_256", [40], [2000], 0),
    ("64_128", [1, 20], [32000, 8000], 0)])
def test_one_key_takes_nearly_all(name, q, past, at, gap):
    """A key with nearly all of the weight and a value of zero: the norm scales
    up what the others add, 2^-gap of it each. Bound as in
    test_as_exact_as_its_rounding, and in fp16 6 * 2^(gap - 34) noise: a
    probability is off by 2^-34 of the row's largest at most, which is 2^(gap -
    34) of the others' mean (noise weighs each key's value by its own)."""
    w = workload(name, q_lens=q, past_lens=past, rotary_dim=0, num_heads=2, drop_slots=0)
    t, hs = w.tensors, w.head_size
    a = 8.0
    t["query"].view(-1, 2, 2, hs)[..., 0] = a
    t["key"].view(-1, 2, 2, hs)[..., 0] = 0
    t["key_cache"][..., 0] = 0
    for b, p in enumerate(past):
        r = _row(w, b, min(at, p - 1))
        t["key_cache"].view(-1, 2, 2, hs)[r] = 0
        t["key_cache"].view(-1, 2, 2, hs)[r, :, :, 0] = gap * np.log(2.0) * hs ** 0.5 / a
        t["value_cache"].view(-1, 2, w.v_head_size)[r] = 0
    d, out, op = run_gpu(w)
    assert op.error_flags() == 0
    ref = D.run_bits(_numpy(w), w.params, W.dtype_tag(w.dtype))
    got = out.double().cpu().numpy().reshape(ref["out"].shape)
    u = UNIT_ROUNDOFF[w.dtype]
    c = 6 * u * u + 2.0 ** -15 + (6 * 2.0 ** (gap - 34) if w.dtype is torch.float16 else 0.0)
    worst = (np.abs(got - ref["out"]) / (u * np.abs(ref["out"]) + c * ref["noise"])).max()
    rel = np.linalg.norm(got - ref["out"]) / np.linalg.norm(ref["out"])
    print(f"RATIO {name} gap {gap}: {worst:.3f}, relative error {rel:.2e}")
    assert worst <= 1, worst


def test_values_that_come_late():
    """Prompts over contexts of three key tiles whose values arrive long after
    their keys: pages spread over 8 GB a cache, the values' lines and address
    translations out of every cache, the keys just read. The same bits as from
    small caches that are at hand."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 36 GB of device memory")
    n, q, NB = 60, 8, 1 << 18
    w = workload("64_128", q_lens=[q] * n, past_lens=[362 - i % 50 for i in range(n)], num_heads=2, drop_slots=0)
    t = {k: v.cuda() for k, v in w.tensors.items()}
    small = {k: t[k].clone() for k in ("key_cache", "value_cache")}
    op = _op(w)
    for _ in range(5):
        want = op.forward(*_args(t), 0)
    big = {k: torch.zeros(NB, *small[k].shape[1:], dtype=w.dtype, device="cuda") for k in small}
    far = DifferentialAttention(**{**w.params, "num_blocks": NB}, max_seqs=n, max_tokens=n * q, own_slots=True)
    other = torch.zeros(16 << 30, dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(1)
    outs = []
    for r in range(15):
        perm = torch.randperm(NB, generator=g)[:w.num_blocks].cuda()
        for k in big:
            big[k][perm] = small[k]
        bt = torch.where(t["block_table"] >= 0, perm[t["block_table"].clamp(min=0).long()], -1).int()
        s = t["slot_mapping"].long()
        slots = (perm[s // 64] * 64 + s % 64).int()
        other[r::1 << 19] += 1
        other[:1 << 28] += 1
        big["key_cache"][perm].sum()
        outs.append(far.forward(*_args({**t, **big, "block_table": bt, "slot_mapping": slots}), 0))
    assert op.error_flags() == 0 and far.error_flags() == 0
    assert [torch.equal(o, want) for o in outs] == [True] * 15


@pytest.mark.parametrize("kind", ["stream", "handle", "default"])
def test_output_is_memory_of_its_stream(kind):
    """The output that forward allocates belongs to the stream it is given, as
    a torch stream or as a handle: once dropped, its memory is not handed to
    the current stream, which the kernels that still write it do not wait for."""
    w = workload("64_128", q_lens=[1, 40], past_lens=[100, 60], drop_slots=0)
    d, want, op = run_gpu(w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    stream = {"stream": side, "handle": side.cuda_stream, "default": 0}[kind]
    with torch.cuda.stream(torch.cuda.Stream() if kind == "default" else torch.cuda.current_stream()):
        out = op.forward(*_args(d), 1, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        at = out.data_ptr()
        del out
        others = [torch.empty_like(want) for _ in range(64)]
        assert all(o.data_ptr() != at for o in others)


def test_first_call_of_an_operator_on_another_stream():
    """The error word is cleared on the constructor's stream: a first call on
    another stream comes behind that, and what it reports stays."""
    w = workload("64_128", q_lens=[1, 40], past_lens=[100, 60], drop_slots=0)
    w.tensors["slot_mapping"][0] = 10 ** 8
    d = {k: v.cuda() for k, v in w.tensors.items()}
    _op(w).forward(*_args(d), 1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # a tenth of a second, ahead of the fill
    op = _op(w)
    op.forward(*_args(d), 1, stream=side)
    torch.cuda.synchronize()
    assert op.error_flags() == B.PA_DEVERR_SLOT


@pytest.mark.parametrize("what", ["block", "context", "past", "position", "qlen", "slot"])
def test_bad_indices_and_nothing_else(what):
    """What a bad page, length, position or slot changes, exactly: the error
    word, zeros in every row of its sequences, the cache rows of its tokens; the
    other sequences stay within one step of the dtype, 2 u |x|, and 2^-20 of the
    largest output where a decode is cut at other places."""
    w = workload("64_128", q_lens=[1, 1, 20, 30], past_lens=[100, 200, 10, 50], drop_slots=0)
    d0, want, _ = run_gpu(w)
    t, cum = w.tensors, w.tensors["cumseq"].tolist()
    old = {k: t[k].clone() for k in ("key_cache", "value_cache")}
    slots = t["slot_mapping"].clone()
    if what == "block":
        t["block_table"][1, 2], t["block_table"][3, 0] = 10 ** 6, -1
        flag, zero, unwritten = B.PA_DEVERR_BLOCK, [1, 3], []
    elif what == "context":  # (the write has no angles for such positions)
        t["past"][1], t["past"][3] = 10 ** 6, w.max_blocks_per_seq * 64 - 10
        assert t["past"][3] >= w.cos_rows
        flag, zero = B.PA_DEVERR_CONTEXT | B.PA_DEVERR_POSITION, [1, 3]
        unwritten = [1] + list(range(cum[3], cum[4]))
    elif what == "past":
        t["past"][1], t["past"][3] = -5, -40
        flag, zero, unwritten = B.PA_DEVERR_CONTEXT, [1, 3], [1] + list(range(cum[3], cum[4]))
    elif what == "position":
        w.params["cos_rows"] = 150
        flag, zero, unwritten = B.PA_DEVERR_POSITION, [1], [1]
    elif what == "qlen":
        flag, zero, unwritten = B.PA_DEVERR_DECODE_QLEN, [], []
    else:
        t["slot_mapping"][0], t["slot_mapping"][5] = 10 ** 8, -2
        flag, zero, unwritten = B.PA_DEVERR_SLOT, [], [0, 5]
    op = _op(w, own_slots=False)
    d, got, _ = run_gpu(w, op=op, decodes=3 if what == "qlen" else None)
    assert op.error_flags() == flag, hex(op.error_flags())
    for k in old:
        rows = {k2: v.view(w.num_blocks * 64, -1) for k2, v in (("old", old[k].cuda()), ("new", d[k]), ("good", d0[k]))}
        keep = torch.ones(w.num_blocks * 64, dtype=torch.bool, device="cuda")
        for n, s in enumerate(slots.tolist()):
            if n in unwritten:
                assert torch.equal(rows["new"][s], rows["old"][s]), (k, n)
                keep[s] = False
        assert torch.equal(rows["new"][keep], rows["good"][keep]), k
    if what == "slot":  # as if the two tokens had no slot
        t["slot_mapping"][0] = t["slot_mapping"][5] = -1
        _, dropped, op = run_gpu(w, op=_op(w, own_slots=False))
        assert op.error_flags() == 0 and torch.equal(got, dropped)
        want = dropped
    for b in range(4):
        rows, good = got[cum[b]:cum[b + 1]].double(), want[cum[b]:cum[b + 1]].double()
        if b in zero:
            assert (rows == 0).all(), b
        elif what == "qlen" and b == 2:
            assert torch.isnan(rows).all()
        else:
            step = 2 * UNIT_ROUNDOFF[w.dtype] * torch.maximum(rows.abs(), good.abs())
            assert ((rows - good).abs() <= step + 2.0 ** -20 * good.abs().max()).all(), b


@pytest.mark.parametrize("n", [8191, 8192])
def test_thousands_of_sequences(n):
    """Both sides of the number of sequences whose offsets the write keeps in
    shared memory: one token each, and a few prompts behind them."""
    rng = np.random.default_rng(n)
    q = [1] * (n - 3) + [9, 0, 17]
    past = [int(x) for x in rng.integers(0, 20, n)]
    w = workload("64_128", q_lens=q, past_lens=past, num_heads=1, kv_num_heads=1, head_size=16, block_size=16)
    check(w, tokens=list(range(0, 40)) + sorted(rng.choice(n, 300, replace=False).tolist()) + list(range(n - 3, n + 23)))
