"""The cache-page operators on the GPU against the oracle, whole number for
whole number: tables, refcounts, cached lengths, slots, page contents and
error bits, over random pools, calls that make no sense, graphs, streams,
and a serving run together with the attention that reads the pages."""
import numpy as np
import pytest
import torch

from oracle import pages_oracle as O
from paged_latent_attention_cache_gb300 import binding as B
from paged_latent_attention_cache_gb300 import workloads as W
from paged_latent_attention_cache_gb300.api import PagedLatentAttention, PagePool

pytestmark = pytest.mark.gpu


class Pair:
    """One pool twice: on the GPU (`pool`) and as numpy arrays."""

    def __init__(self, seed, nb=64, bs=16, ns=12, mb=10, widths=(48, 16, 1024), fill=0.5, share=True):
        rng = self.rng = np.random.default_rng(seed)
        self.bs, self.nb, self.ns, self.mb = bs, nb, ns, mb
        self.caches = [rng.integers(0, 256, size=(nb, bs, w)).astype(np.uint8) for w in widths]
        self.table = np.full((ns, mb), -1, np.int32)
        self.past = np.zeros(ns, np.int32)
        free = list(rng.permutation(nb))
        for b in range(ns):
            if rng.random() > fill or not free:
                continue
            n = min(int(rng.integers(1, mb + 1)), len(free))
            self.table[b, :n] = [free.pop() for _ in range(n)]
            self.past[b] = (n - 1) * bs + rng.integers(0, bs + 1)
        if share:  # some rows start with another row's pages, as after a fork
            full = [b for b in range(ns) if self.past[b] >= bs]
            empty = [b for b in range(ns) if self.past[b] == 0 and (self.table[b] < 0).all()]
            for c, p in zip(empty[::2], full):
                n = self.past[p] // bs
                self.table[c, :n] = self.table[p, :n]
                self.past[c] = n * bs
        self.ref = np.bincount(self.table[self.table >= 0], minlength=nb).astype(np.int32)
        self.upload()

    def upload(self):
        d = lambda a: torch.from_numpy(a.copy()).cuda()
        self.pool = PagePool([d(c) for c in self.caches], block_size=self.bs,
                             block_table=d(self.table), past=d(self.past), refcount=d(self.ref))

    def ints(self, a):
        return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()

    def check(self, err):
        p = self.pool
        torch.cuda.synchronize()
        assert p.error_flags() == err, (hex(p.error_flags()), hex(err))
        assert np.array_equal(p.block_table.cpu().numpy(), self.table)
        assert np.array_equal(p.past.cpu().numpy(), self.past)
        assert np.array_equal(p.refcount.cpu().numpy(), self.ref)
        for a, b in zip(p.caches, self.caches):
            assert np.array_equal(a.cpu().numpy(), b)
        p.reset_error_flags()


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("with_rows", [False, True])
def test_copy_random(seed, with_rows):
    s = Pair(seed, nb=[2, 7, 64, 300, 1000, 64][seed], bs=[16, 32, 16, 16, 16, 128][seed])
    perm = s.rng.permutation(s.nb)
    n = s.nb // 2
    src, dst = perm[:n], perm[n:2 * n]
    rows = s.rng.integers(0, s.bs + 1, size=n) if with_rows else None
    s.pool.copy(s.ints(src), s.ints(dst), None if rows is None else s.ints(rows))
    s.check(O.copy(s.caches, src, dst, rows, s.bs))


@pytest.mark.parametrize("src,dst,rows", [
    ([1, 2, 3], [5, 5, 6], None),          # a destination twice: the first pair
    ([1, 5, 7], [5, 6, 7], None),          # a source that is written; a page onto itself
    ([1, 2], [2, 1], None),                # a swap
    ([-1, 64, 3, 4], [5, 6, -2, 99], None),
    ([1, 2, 3], [9, 10, 11], [17, -1, 4]),
    ([3, 3, 3], [9, 10, 11], [0, 16, 1]),
    ([2, 1, 4], [9, 9, 2], None),          # the refused pair's destination still counts
])
def test_copy_conflicts(src, dst, rows):
    s = Pair(3)
    s.pool.copy(s.ints(src), s.ints(dst), None if rows is None else s.ints(rows))
    s.check(O.copy(s.caches, src, dst, rows, s.bs))


@pytest.mark.parametrize("n", [1, 63, 64, 65, 300])
def test_copy_conflicts_by_count(n):
    """Random pairs with every kind of conflict, on both sides of the number
    up to which a copy is one kernel."""
    s = Pair(n, nb=400)
    src, dst = s.rng.integers(-1, 401, size=n), s.rng.integers(-1, 401, size=n)
    rows = s.rng.integers(-1, 18, size=n)
    s.pool.copy(s.ints(src), s.ints(dst), s.ints(rows))
    s.check(O.copy(s.caches, src, dst, rows, s.bs))


def test_copy_many_caches_and_page_sizes():
    """More caches than one launch takes, pages from 256 bytes to 96 KB."""
    widths = [16 * (1 + i % 7) for i in range(150)] + [1536 * 4]
    s = Pair(5, nb=40, widths=widths)
    src, dst = np.arange(0, 40, 2), np.arange(1, 40, 2)
    rows = s.rng.integers(0, 17, size=20)
    s.pool.copy(s.ints(src), s.ints(dst), s.ints(rows))
    s.check(O.copy(s.caches, src, dst, rows, s.bs))


@pytest.mark.parametrize("seed", range(8))
def test_fork_random(seed):
    s = Pair(seed, nb=[64, 64, 400, 64, 40, 600, 64, 64][seed], ns=[12, 12, 300, 12, 12, 40, 5, 12][seed],
             mb=[10, 10, 10, 40, 10, 50, 10, 1][seed])
    n = int(s.rng.integers(1, s.ns + 1))
    parents, children = s.rng.integers(0, s.ns, size=n), s.rng.permutation(s.ns)[:n]
    s.pool.fork(s.ints(parents), s.ints(children))
    s.check(O.fork(s.caches, s.table, s.past, s.ref, parents, children, s.bs))


def _forkable():
    s = Pair(1, share=False, fill=0.0)
    s.table[0, :4], s.past[0] = [7, 3, 9, 11], 3 * 16 + 5
    s.table[1, :2], s.past[1] = [20, 21], 32
    s.table[2, :10], s.past[2] = np.arange(30, 40), 160
    s.ref = np.bincount(s.table[s.table >= 0], minlength=s.nb).astype(np.int32)
    return s


@pytest.mark.parametrize("parents,children", [
    ([0, 0, 0, 1, 2], [4, 5, 6, 7, 8]),
    ([0, 1], [5, 5]),           # a child twice
    ([0, 5], [5, 6]),           # a parent that is a child
    ([0], [0]), ([0], [1]),     # itself; a child that holds pages
    ([3], [4]),                 # an empty parent
    ([0, -1, 12, 0], [4, 5, 6, 12]),
    ([9, 0], [4, 4]),
])
def test_fork_conflicts(parents, children):
    s = _forkable()
    s.upload()
    s.pool.fork(s.ints(parents), s.ints(children))
    s.check(O.fork(s.caches, s.table, s.past, s.ref, parents, children, s.bs))


@pytest.mark.parametrize("break_it", ["past_negative", "past_long", "page_range", "page_free", "full_pool"])
def test_fork_broken_state(break_it):
    s = _forkable()
    if break_it == "past_negative":
        s.past[0] = -3
    elif break_it == "past_long":
        s.past[0] = 161
    elif break_it == "page_range":
        s.table[0, 1] = 64
    elif break_it == "page_free":
        s.ref[9] = 0
    else:
        s.ref[:] = np.maximum(s.ref, 1)
        s.ref[50] = 0  # one page left for two forks
    s.upload()
    parents, children = [0, 1, 0], [4, 5, 6]
    s.pool.fork(s.ints(parents), s.ints(children))
    s.check(O.fork(s.caches, s.table, s.past, s.ref, parents, children, s.bs))


@pytest.mark.parametrize("seed", range(4))
def test_free_random(seed):
    s = Pair(seed, ns=40, nb=200, mb=300 if seed == 3 else 10, fill=0.8)
    seqs = s.rng.integers(0, s.ns, size=s.ns)  # some twice
    s.pool.free(s.ints(seqs))
    s.check(O.free(s.table, s.past, s.ref, seqs))
    s.pool.free(s.ints(seqs))
    s.check(0)


def test_free_broken_state():
    s = _forkable()
    s.table[0, 1], s.table[1, 0] = 64, -7
    s.ref[9] = 0
    s.upload()
    seqs = [0, 1, -1, 12, 2]
    s.pool.free(s.ints(seqs))
    s.check(O.free(s.table, s.past, s.ref, seqs))


@pytest.mark.parametrize("seed", range(10))
def test_reserve_random(seed):
    s = Pair(seed, nb=[64, 64, 64, 600, 600, 5000, 33, 64, 2000, 64][seed],
             ns=[12, 1, 12, 300, 40, 700, 12, 12, 3, 12][seed], mb=[10, 10, 10, 10, 64, 10, 10, 10, 500, 10][seed],
             bs=[16, 16, 32, 16, 16, 16, 16, 128, 16, 16][seed])
    room = s.mb * s.bs - s.past
    q = np.minimum(s.rng.integers(0, 3 * s.bs, size=s.ns), room)
    if seed == 8:
        q = room
    cum = np.concatenate([[0], np.cumsum(q)])
    pad = 5 if seed % 2 else 0
    T = int(cum[-1]) + pad
    slots = torch.full((T,), 12345, dtype=torch.int32, device="cuda")
    s.pool.reserve(s.ints(cum), slots)
    err, want = O.reserve(s.table, s.past, s.ref, cum, T, s.bs)
    assert np.array_equal(slots.cpu().numpy(), want)
    s.check(err)


@pytest.mark.parametrize("tokens", [24575, 24576, 24577, 60000])
def test_reserve_many_tokens(tokens):
    """Both sides of the number of tokens up to which one kernel does it all;
    the pool gives out before the last sequence."""
    s = Pair(7, nb=4000, ns=40, mb=200, fill=0.0, share=False, widths=(16,))
    q = np.full(40, tokens // 40)
    q[7], q[20] = 0, q[20] + q[7]
    q[39] += tokens - q.sum()
    cum = np.concatenate([[0], np.cumsum(q)])
    if tokens == 60000:
        s.ref[:1000] = 1  # held by nobody's row, but held
        s.upload()
    slots = torch.full((tokens,), 12345, dtype=torch.int32, device="cuda")
    s.pool.reserve(s.ints(cum), slots)
    err, want = O.reserve(s.table, s.past, s.ref, cum, tokens, s.bs)
    assert np.array_equal(slots.cpu().numpy(), want)
    assert (err == O.POOL) == (tokens == 60000)
    s.check(err)


@pytest.mark.parametrize("break_it", ["past", "long", "hole", "shared", "range", "free", "cumseq", "start", "far"])
def test_reserve_broken_state(break_it):
    s = _forkable()
    s.past[2] = 150
    cum = np.array([0, 30, 47, 50] + [50] * 8 + [60])
    if break_it == "past":
        s.past[0] = -1
    elif break_it == "long":
        s.past[0] = 140
    elif break_it == "hole":
        s.table[0, 3] = -1
    elif break_it == "shared":
        s.ref[11] = 2
    elif break_it == "range":
        s.table[0, 3] = 64
    elif break_it == "free":
        s.ref[11] = 0
    elif break_it == "cumseq":
        cum[1] = 55
    elif break_it == "start":
        cum[0] = -2
    else:
        cum[-1] = 1000
    s.upload()
    T = 60
    slots = torch.full((T,), 12345, dtype=torch.int32, device="cuda")
    s.pool.reserve(s.ints(cum), slots)
    err, want = O.reserve(s.table, s.past, s.ref, cum, T, s.bs)
    got = slots.cpu().numpy()
    if break_it != "cumseq":
        assert np.array_equal(got, want)
    else:  # overlapping sequences: which one a token falls in is open, but its slot is one of theirs
        assert np.isin(got // s.bs, [-1] + s.table[s.table >= 0].tolist()).all()
    s.check(err)


@pytest.mark.parametrize("seed", range(6))
def test_compact_random(seed):
    s = Pair(seed, nb=[64, 1, 1000, 64, 20000, 64][seed], ns=[12, 1, 60, 12, 40, 12][seed],
             mb=[10, 1, 10, 10, 300, 10][seed], fill=[0.5, 1.0, 0.7, 0.0, 0.9, 1.0][seed],
             widths=(16,) if seed == 4 else (48, 16, 1024))
    live = s.pool.compact()
    err, want = O.compact(s.caches, s.table, s.ref)
    s.check(err)
    assert int(live.item()) == want
    s.pool.compact()  # a compact pool stays as it is
    s.check(0)


def test_compact_broken_table():
    s = _forkable()
    s.table[5, 0], s.table[5, 1], s.table[6, 0] = 64, -9, 60  # none of the pool; a free page
    s.upload()
    s.pool.compact()
    err, _ = O.compact(s.caches, s.table, s.ref)
    s.check(err)


def test_graph_replay_and_streams():
    """free + fork + reserve captured once and replayed on another stream:
    every replay computes from the state it finds."""
    s = _forkable()
    s.upload()
    parents, children = s.ints([0, 0, 1]), s.ints([4, 5, 6])
    cum = np.array([0, 0, 0, 0, 0, 20, 40, 60] + [60] * 5)
    cum_d, slots = s.ints(cum), torch.zeros(60, dtype=torch.int32, device="cuda")

    def step():
        s.pool.free(children)
        s.pool.fork(parents, children)
        s.pool.reserve(cum_d, slots)

    def oracle():
        O.free(s.table, s.past, s.ref, [4, 5, 6])
        e = O.fork(s.caches, s.table, s.past, s.ref, [0, 0, 1], [4, 5, 6], s.bs)
        e2, want = O.reserve(s.table, s.past, s.ref, cum, 60, s.bs)
        return e | e2, want

    step()
    err, want = oracle()
    torch.cuda.synchronize()
    assert np.array_equal(slots.cpu().numpy(), want)
    s.check(err)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    side = torch.cuda.Stream()
    for k in range(3):
        s.table[0, 2] = 50 + k  # the state moves on between replays
        s.ref[:] = np.bincount(s.table[s.table >= 0], minlength=s.nb)
        s.pool.block_table.copy_(torch.from_numpy(s.table))
        s.pool.refcount.copy_(torch.from_numpy(s.ref))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        err, want = oracle()
        assert np.array_equal(slots.cpu().numpy(), want)
        s.check(err)


def test_pool_refuses_bad_tensors():
    c = torch.zeros(8, 16, 32, dtype=torch.uint8, device="cuda")
    pool = PagePool([c], block_size=16, max_seqs=4, max_blocks_per_seq=3)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    for bad in (lambda: pool.copy(i32(1).long(), i32(2)), lambda: pool.copy(i32(1), i32(2, 3)),
                lambda: pool.copy(i32(1).cpu(), i32(2)), lambda: pool.fork(i32(1, 2), i32(3)),
                lambda: pool.free(i32(1, 2, 3, 4)[::2]), lambda: pool.reserve(i32(0, 1), i32(0)),
                lambda: pool.copy(i32(1), i32(2), i32(3, 4)),
                lambda: PagePool([c.permute(0, 2, 1)], block_size=32, max_seqs=1, max_blocks_per_seq=1),
                lambda: PagePool([c], block_size=32, max_seqs=1, max_blocks_per_seq=1),
                lambda: PagePool([c], block_size=16),
                lambda: PagePool([c, c.cpu()], block_size=16, max_seqs=1, max_blocks_per_seq=1),
                lambda: PagePool([c[:, :, :8]], block_size=16, max_seqs=1, max_blocks_per_seq=1),
                lambda: PagePool([torch.zeros(8, 16, 8, dtype=torch.uint8, device="cuda")], block_size=16,
                                 max_seqs=1, max_blocks_per_seq=1)):
        with pytest.raises(B.PaError):
            bad()


def test_serving_run_with_attention():
    """Prompts, forks, tokens and a compaction, all addressed by the pool: the
    forked sequences answer exactly as their parent, and compaction changes no
    output bit."""
    H, bs, nb, ns, mb = 8, 16, 64, 6, 8
    g = torch.Generator().manual_seed(0)
    cos, sin = (t.cuda() for t in W.rope_tables(mb * bs, 64, torch.bfloat16))
    cache = torch.randn(nb, bs, 1, 192, generator=g).bfloat16().cuda()
    pool = PagePool([cache], block_size=bs, max_seqs=ns, max_blocks_per_seq=mb)
    op = PagedLatentAttention(dtype=torch.bfloat16, num_heads=H, head_size=192, v_head_size=128,
                              rotary_offset=128, rotary_dim=64, cos_rows=mb * bs, block_size=bs,
                              num_blocks=nb, max_blocks_per_seq=mb, scale=192 ** -0.5,
                              max_seqs=ns, max_tokens=256)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")

    def rows(n, w, seed):
        return torch.randn(n, w, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()

    def attend(q_lens, query, key, decodes):
        cum = i32([0] + list(np.cumsum(q_lens)))
        slots = pool.reserve(cum, torch.empty(int(sum(q_lens)), dtype=torch.int32, device="cuda"))
        out = op.forward(query, key, cache, cos, sin, cum, pool.past, pool.block_table, slots, decodes)
        pool.past += cum[1:] - cum[:-1]
        return out

    attend([37, 64, 5, 0, 0, 0], rows(106, H * 192, 1), rows(106, 192, 2), 0)
    pool.free(i32([1]))  # its four pages leave a hole below sequence 2's
    pool.fork(i32([0, 0, 2]), i32([3, 4, 5]))
    pool.fork(i32([2]), i32([1]))
    one = lambda seed, w: rows(3, w, seed)
    q3, k3 = one(3, H * 192), one(4, 192)
    pick = [0, 2, 1, 0, 0, 1]  # sequences 0, 3, 4 say the same, as do 2, 5; 1 differs
    out = attend([1] * 6, q3[pick].contiguous(), k3[pick].contiguous(), 6)
    assert pool.error_flags() == 0 and op.error_flags() == 0
    assert torch.equal(out[0], out[3]) and torch.equal(out[0], out[4]) and torch.equal(out[2], out[5])
    assert not torch.equal(out[1], out[2])

    def read():
        o = torch.zeros(6, H * 128, dtype=torch.bfloat16, device="cuda")
        op.decode(q3[pick].contiguous(), cache, cos, sin, i32(range(7)), pool.past - 1,
                  pool.block_table, o)
        return o

    before = read()
    pool.free(i32([0]))
    live = int(pool.compact().item())
    assert int(pool.block_table.max().item()) == live - 1
    after = read()
    assert torch.equal(before[1:], after[1:]) and pool.error_flags() == 0


def test_one_page_in_many_caches():
    """A pool of a single page: nothing can move, in any number of caches."""
    caches = [torch.arange(16 * 16, dtype=torch.uint8, device="cuda").view(1, 16, 16) for _ in range(130)]
    pool = PagePool(caches, block_size=16, max_seqs=2, max_blocks_per_seq=1)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    slots = pool.reserve(i32(0, 5, 5), torch.empty(5, dtype=torch.int32, device="cuda"))
    assert slots.tolist() == [0, 1, 2, 3, 4]
    assert pool.compact().tolist() == [1]
    pool.copy(i32(0), i32(0))
    assert pool.error_flags() == 0 and pool.block_table.tolist() == [[0], [-1]]
    pool.past += i32(5, 0)
    pool.fork(i32(0), i32(1))
    assert pool.error_flags() == B.PA_DEVERR_POOL
    pool.free(i32(0, 1))
    assert pool.compact().tolist() == [0] and pool.refcount.tolist() == [0]
    assert all(torch.equal(c, caches[0]) for c in caches)


def test_tiny_calls_in_a_row():
    """Pools so small that nearly every warp of the bookkeeping has nothing to
    look at: a long run of reserve, compact and free calls, none of which the
    host waits for."""
    s = Pair(11, nb=3, ns=2, mb=2, widths=(16,), fill=0.0, share=False)
    cum = np.array([0, 17, 20])
    seqs = s.ints([0])
    slots = [torch.full((21,), 12345, dtype=torch.int32, device="cuda") for _ in range(60)]
    cum_d, wants, lives = s.ints(cum), [], []
    for t in slots:
        s.pool.reserve(cum_d, t)
        s.pool.free(seqs)
        lives.append(s.pool.compact().clone())
        s.pool.reserve(cum_d, t)
    err = 0
    for _ in slots:
        err |= O.reserve(s.table, s.past, s.ref, cum, 21, s.bs)[0]
        err |= O.free(s.table, s.past, s.ref, [0])
        e, live = O.compact(s.caches, s.table, s.ref)
        e2, want = O.reserve(s.table, s.past, s.ref, cum, 21, s.bs)
        err |= e | e2
        wants.append((live, want))
    s.check(err)
    for t, n, (live, want) in zip(slots, lives, wants):
        assert np.array_equal(t.cpu().numpy(), want) and int(n.item()) == live


@pytest.mark.parametrize("handle", [False, True])
def test_first_call_on_another_stream(handle):
    """The constructor fills table, lengths and refcounts on the current stream;
    a first call on another stream comes behind that, however late it is."""
    cache = torch.zeros(64, 16, 16, dtype=torch.uint8, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    cum, slots = i32([0, 20, 25]), torch.zeros(25, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    warm = PagePool([cache], block_size=16, max_seqs=2, max_blocks_per_seq=4)
    warm.reserve(cum, slots, stream=side)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # a tenth of a second, ahead of the fills
    pool = PagePool([cache], block_size=16, max_seqs=2, max_blocks_per_seq=4)
    pool.reserve(cum, slots, stream=side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert pool.error_flags() == 0
    assert pool.block_table.tolist() == [[0, 1, -1, -1], [2, -1, -1, -1]]
    assert pool.refcount.tolist() == [1, 1, 1] + [0] * 61
    assert slots.tolist() == list(range(20)) + list(range(32, 37))
    graph = torch.cuda.CUDAGraph()
    late = PagePool([cache], block_size=16, max_seqs=2, max_blocks_per_seq=4)
    with torch.cuda.graph(graph):  # its first call captured
        late.reserve(cum, slots)
    graph.replay()
    torch.cuda.synchronize()
    assert late.block_table.tolist() == pool.block_table.tolist() and late.error_flags() == 0


def test_pool_refuses_empty_caches():
    """Caches without a page, a row or a dimension for them."""
    zeros = lambda *shape: torch.zeros(*shape, dtype=torch.uint8, device="cuda")
    for bad in (zeros(0, 16, 16), zeros(8, 16, 0), zeros(8), zeros(8, 0, 16), zeros(())):
        with pytest.raises(B.PaError):
            PagePool([bad], block_size=16, max_seqs=1, max_blocks_per_seq=1)


@pytest.mark.parametrize("seed", range(3))
def test_beam_steps_between_two_sets_of_rows(seed):
    """Beams that go on from one another, step by step: each forks into the
    other set of rows, the first set is freed, and every beam gets a token."""
    beams, steps = 4, 12
    s = Pair(seed, nb=80, ns=2 * beams, mb=6, fill=0.0, share=False)
    s.table[:beams, :2] = np.arange(2 * beams).reshape(beams, 2)
    s.past[:beams] = s.rng.integers(17, 33, size=beams)
    s.ref = np.bincount(s.table[s.table >= 0], minlength=s.nb).astype(np.int32)
    s.upload()
    here = 0
    for _ in range(steps):
        there = beams - here
        parents, children = here + s.rng.integers(0, beams, beams), there + np.arange(beams)
        rows = here + np.arange(beams)
        q = np.zeros(2 * beams, int)
        q[children] = 1
        cum = np.concatenate([[0], np.cumsum(q)])
        slots = torch.zeros(beams, dtype=torch.int32, device="cuda")
        s.pool.fork(s.ints(parents), s.ints(children))
        s.pool.free(s.ints(rows))
        s.pool.reserve(s.ints(cum), slots)
        err = O.fork(s.caches, s.table, s.past, s.ref, parents, children, s.bs)
        err |= O.free(s.table, s.past, s.ref, rows)
        e, want = O.reserve(s.table, s.past, s.ref, cum, beams, s.bs)
        assert err | e == 0 and np.array_equal(slots.cpu().numpy(), want)
        s.past[children] += 1
        s.pool.past += s.ints(q)
        s.check(0)
        here = there


@pytest.mark.parametrize("ns,long", [(4096, False), (4097, False), (4097, True), (9000, True), (20000, False)])
def test_thousands_of_sequences(ns, long):
    """More sequences than their offsets' place in shared memory, with the slots
    filled by the cluster (up to 24576 tokens) and apart, pages for half of the
    needs; forks, and all freed."""
    s = Pair(ns, nb=2 * ns, ns=ns, mb=3, fill=0.3, widths=(16,))
    q = np.where(s.rng.random(ns) < 0.9, 1, 0)
    if long:
        q *= s.rng.integers(1, 20, size=ns)
    q = np.minimum(q, s.mb * s.bs - s.past)
    cum = np.concatenate([[0], np.cumsum(q)])
    T = int(cum[-1]) + 3
    lack = int((-(-(s.past + q) // s.bs) - (s.table >= 0).sum(1)).clip(0).sum())
    free = np.flatnonzero(s.ref == 0)
    s.ref[s.rng.permutation(free)[lack // 2:]] = 1  # held by nobody's row, but held
    s.upload()
    slots = torch.full((T,), 12345, dtype=torch.int32, device="cuda")
    s.pool.reserve(s.ints(cum), slots)
    err, want = O.reserve(s.table, s.past, s.ref, cum, T, s.bs)
    assert np.array_equal(slots.cpu().numpy(), want) and err & O.POOL and (want >= 0).sum() > T // 4
    s.check(err)
    parents, children = s.rng.integers(0, ns, size=ns), s.rng.permutation(ns)
    s.pool.fork(s.ints(parents), s.ints(children))
    s.check(O.fork(s.caches, s.table, s.past, s.ref, parents, children, s.bs))
    seqs = s.rng.permutation(ns)
    s.pool.free(s.ints(seqs))
    s.check(O.free(s.table, s.past, s.ref, seqs))


def test_first_call_captured_by_its_handle():
    """A capture of the given stream, while another one is current, takes no
    wait for the constructor's event, which lies outside."""
    cache = torch.zeros(64, 16, 16, dtype=torch.uint8, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    cum, slots = i32([0, 20, 25]), torch.zeros(25, dtype=torch.int32, device="cuda")
    PagePool([cache], block_size=16, max_seqs=2, max_blocks_per_seq=4).reserve(cum, slots)
    pool = PagePool([cache], block_size=16, max_seqs=2, max_blocks_per_seq=4)
    slots.fill_(7)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        graph.capture_begin()
    pool.reserve(cum, slots, stream=side.cuda_stream)
    with torch.cuda.stream(side):
        graph.capture_end()
    assert slots.tolist() == [7] * 25
    graph.replay()
    torch.cuda.synchronize()
    assert slots.tolist() == list(range(20)) + list(range(32, 37)) and pool.error_flags() == 0
