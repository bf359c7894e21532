"""The cache-page operators and differential attention, as calls that can be timed and compared.

Two families over the paged caches:

* page operators (``api.PagePool``): copying pages, forking sequences, freeing them, reserving pages
  for new tokens and compacting the pool, over every layer's cache at once;
* differential attention (``api.DifferentialAttention``): the write of new rows and the read of one
  new token per sequence (decode) or of whole chunks (prefill).

``own`` false computes them with elementary torch operations, ``own`` true calls the framework.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda"


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one request's shared prefix copied before it is edited: few small pages, latency counts
        {"name": "copy_few", "op": "copy", "layers": 4, "width": 192, "vwidth": 0, "bs": 16, "blocks": 1024, "n": 8,
         "rows": False},
        # a pool of 576-wide rows: many whole and partly filled pages moved in 16 layers
        {"name": "copy_many", "op": "copy", "layers": 16, "width": 576, "vwidth": 0, "bs": 64, "blocks": 2048, "n": 768,
         "rows": True},
        # one step of a small beam search: the old beams are freed, two prompts fork two beams each
        {"name": "fork_few", "op": "fork", "layers": 4, "width": 192, "vwidth": 0, "bs": 16, "parents": 2, "beams": 2,
         "lo": 100, "hi": 1000},
        # parallel sampling over a full batch: 64 prompts of 1024..8192 tokens, four samples each
        {"name": "fork_many", "op": "fork", "layers": 8, "width": 576, "vwidth": 0, "bs": 64, "parents": 64, "beams": 4,
         "lo": 1024, "hi": 8192},
        # a small pool compacted after most of its sequences ended
        {"name": "compact_small", "op": "compact", "layers": 4, "width": 192, "vwidth": 0, "bs": 16, "blocks": 512,
         "seqs": 8, "live": 0.5},
        # a large one: 40 % of 8192 pages live and scattered
        {"name": "compact_large", "op": "compact", "layers": 8, "width": 576, "vwidth": 0, "bs": 64, "blocks": 8192,
         "seqs": 48, "live": 0.4},
        # one step of continuous batching, small: finished rows freed, new prompts and tokens get pages and slots
        {"name": "step_small", "op": "step", "bs": 16, "blocks": 1024, "seqs": 16, "ended": 2, "prompt": 100, "hi": 500},
        # the same for 512 rows on a pool of 131072 pages, contexts up to 32768
        {"name": "step_large", "op": "step", "bs": 16, "blocks": 131072, "seqs": 512, "ended": 64, "prompt": 1500,
         "hi": 6000},
        # two short conversations, one token each: latency counts
        {"name": "decode_few", "op": "attend", "dtype": "fp16", "heads": 8, "kv": 4, "hs": 64, "vhs": 128, "bs": 16,
         "seqs": 2, "q": 1, "lo": 300, "hi": 1000, "depth": 1, "window": -1},
        # a full decode batch of 1024..8192 cached tokens
        {"name": "decode_batch", "op": "attend", "dtype": "bf16", "heads": 16, "kv": 8, "hs": 128, "vhs": 256, "bs": 64,
         "seqs": 32, "q": 1, "lo": 1024, "hi": 8192, "depth": 12, "window": -1},
        # short prompt chunks after some context
        {"name": "prefill_chunk", "op": "attend", "dtype": "fp16", "heads": 8, "kv": 8, "hs": 64, "vhs": 128, "bs": 16,
         "seqs": 2, "q": 250, "lo": 350, "hi": 1500, "depth": 3, "window": -1},
        # long prompts: 4096 new tokens on up to 4096 cached ones
        {"name": "prefill_long", "op": "attend", "dtype": "bf16", "heads": 16, "kv": 4, "hs": 128, "vhs": 256, "bs": 128,
         "seqs": 2, "q": 4096, "lo": 4096, "hi": 8192, "depth": 20, "window": -1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["copy", "fork", "compact", "step", "attend", "attend", "attend"])
    bs = rng.choice([16, 32, 64, 128])
    if op == "attend":
        hs, vhs = rng.choice([(64, 128), (128, 256), (64, 64), (128, 128), (96, 192), (48, 80), (32, 64)])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 3, 4, 8])
        heads = heads if heads <= 32 else 2 * kv
        c = {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "heads": heads, "kv": kv, "hs": hs, "vhs": vhs, "bs": bs,
             "depth": rng.randrange(24), "window": rng.choice([-1, -1, _log(rng, 16, 4096)])}
        if rng.random() < 0.6:
            hi = _log(rng, 64, 65536)
            seqs = _log(rng, 1, max(1, min(64, 131072 // hi)))
            return {**c, "seqs": seqs, "q": 1, "lo": max(1, int(hi * rng.uniform(0.05, 1.0))), "hi": hi}
        q = _log(rng, 2, 2048)
        hi = q + rng.randrange(2049)
        return {**c, "seqs": rng.randint(1, 4), "q": q, "lo": q, "hi": hi}
    layers = rng.randint(1, 16)
    width, vwidth = rng.choice([(192, 0), (576, 0), (1024, 1024), (2048, 2048), (512, 1024)])
    pool = (1 << 31) // (layers * bs * (width + vwidth) * 2)  # pages of at most 2 GB in all
    if op == "copy":
        blocks = max(16, min(4096, pool))
        return {"op": op, "layers": layers, "width": width, "vwidth": vwidth, "bs": bs, "blocks": blocks,
                "n": _log(rng, 1, blocks // 4), "rows": rng.random() < 0.5}
    if op == "fork":
        parents, beams = _log(rng, 1, 48), rng.randint(1, 5)
        hi = max(bs + 1, min(8192, bs * (pool // (2 * parents))))
        return {"op": op, "layers": layers, "width": width, "vwidth": vwidth, "bs": bs, "parents": parents,
                "beams": beams, "lo": max(1, hi // 8), "hi": hi}
    if op == "compact":
        blocks = _log(rng, 64, max(65, min(8192, pool)))
        return {"op": op, "layers": layers, "width": width, "vwidth": vwidth, "bs": bs, "blocks": blocks,
                "seqs": rng.randint(2, 32), "live": round(rng.uniform(0.1, 0.9), 3)}
    seqs = _log(rng, 4, 512)
    prompt, hi = _log(rng, 16, 1500), _log(rng, 64, 6000)
    return {"op": op, "bs": bs, "blocks": 64 + seqs * (2 + (hi + 2 * prompt) // bs), "seqs": seqs,
            "ended": max(1, seqs // rng.randint(2, 16)), "prompt": prompt, "hi": hi}


# ------------------------------------------------------------------------------------------ inputs

def _spread(rng, lo, hi, n):
    """n whole numbers evenly spread over [lo, hi], hi among them, in random order."""
    return rng.permutation(np.linspace(hi, lo, n + 1)[:n].round().astype(np.int64))


def _deal(pages, ctx_pages, mb, rows):
    """A block table whose row r holds the next ctx_pages[r] of `pages`."""
    table = np.full((rows, mb), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(ctx_pages):
        table[r, :n] = pages[at:at + n]
        at += n
    return table


def _dev(a, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(a)).to(device=DEV, dtype=dtype)


def _pools(c, blocks, gen):
    """Cached rows N(0, 0.5^2) of all layers: one tensor for the keys and, where the layout has
    them, one for the values."""
    return [torch.empty(c["layers"], blocks, c["bs"], w, dtype=torch.bfloat16, device=DEV).normal_(0.0, 0.5, generator=gen)
            for w in (c["width"], c["vwidth"]) if w]


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return {"copy": _prepare_copy, "fork": _prepare_fork, "compact": _prepare_compact, "step": _prepare_step,
            "attend": _prepare_attend}[case["op"]](case, rng, gen)


def _state(c, caches, table, past, ref, **more):
    s = {"case": c, "caches": caches, "table": _dev(table), "past": _dev(past), "ref": _dev(ref), **more}
    if own:
        from paged_latent_attention_cache_gb300.api import PagePool
        s["pool"] = PagePool([layer for t in caches for layer in t], block_size=c["bs"], block_table=s["table"],
                             past=s["past"], refcount=s["ref"])
    return s


def _prepare_copy(c, rng, gen):
    perm = rng.permutation(c["blocks"])
    src, dst = perm[:c["n"]], perm[c["n"]:2 * c["n"]]
    rows = rng.integers(1, c["bs"] + 1, size=c["n"]) if c["rows"] else None
    none = np.full((1, 1), -1, dtype=np.int32)
    return _state(c, _pools(c, c["blocks"], gen), none, [0], np.zeros(c["blocks"]), src=_dev(src), dst=_dev(dst),
                  rows=None if rows is None else _dev(rows))


def _prepare_fork(c, rng, gen):
    ctx = _spread(rng, c["lo"], c["hi"], c["parents"])
    pages = -(-ctx // c["bs"])
    kids = c["parents"] * c["beams"]
    blocks, mb = int(pages.sum()) + kids + kids // 4 + 8, int(pages.max()) + 1
    perm = rng.permutation(blocks)
    table = _deal(perm, pages, mb, c["parents"] + kids)
    past = np.concatenate([ctx, np.zeros(kids, dtype=np.int64)])
    ref = np.bincount(table[table >= 0], minlength=blocks)
    return _state(c, _pools(c, blocks, gen), table, past, ref,
                  parents=_dev(np.repeat(np.arange(c["parents"]), c["beams"])),
                  children=_dev(c["parents"] + np.arange(kids)))


def _prepare_compact(c, rng, gen):
    live = max(c["seqs"], int(c["blocks"] * c["live"]))
    mb = 2 * (live // c["seqs"]) - 1  # sequences of 1..mb pages
    pages = rng.permutation(np.linspace(1, mb, c["seqs"]).astype(np.int64))
    table = _deal(rng.permutation(c["blocks"]), pages, mb, 2 * c["seqs"])
    table[c["seqs"]:, :] = table[:c["seqs"], :]  # every sequence forked once: half of its pages shared
    table[c["seqs"]:, (mb + 1) // 2:] = -1
    ref = np.bincount(table[table >= 0], minlength=c["blocks"])
    past = (table >= 0).sum(1) * c["bs"]
    s = _state(c, _pools(c, c["blocks"], gen), table, past, ref)
    s["table0"], s["ref0"], s["moved"] = s["table"].clone(), s["ref"].clone(), _moved(ref)
    return s


def _moved(ref):
    live = int((ref > 0).sum())
    return int((ref[live:] > 0).sum())


def _prepare_step(c, rng, gen):
    n, bs = c["seqs"], c["bs"]
    past = _spread(rng, 1, c["hi"], n)
    ended = np.sort(rng.choice(n, size=c["ended"], replace=False))
    fresh = _spread(rng, 1, 2 * c["prompt"], c["ended"])
    q = np.ones(n, dtype=np.int64)
    q[ended] = fresh
    pages = -(-past // bs)
    mb, blocks = max(c["hi"], 2 * c["prompt"]) // bs + 2, c["blocks"]
    table = _deal(rng.permutation(blocks), pages, mb, n)
    ref = np.bincount(table[table >= 0], minlength=blocks)
    cumseq = np.concatenate([[0], np.cumsum(q)])
    none = torch.zeros(1, blocks, bs, 8, dtype=torch.bfloat16, device=DEV)
    return _state(c, [none], table, past, ref, ended=_dev(ended), cumseq=_dev(cumseq), tokens=int(q.sum()),
                  slots=torch.empty(int(q.sum()), dtype=torch.int32, device=DEV))


def _prepare_attend(c, rng, gen):
    dt = DTYPES[c["dtype"]]
    H, kv, hs, vhs, bs, n = c["heads"], c["kv"], c["hs"], c["vhs"], c["bs"], c["seqs"]
    ctx = _spread(rng, c["lo"], c["hi"], n)
    q = np.full(n, c["q"], dtype=np.int64)
    pages = -(-ctx // bs)
    blocks = int(pages.sum()) + 4
    table = _deal(rng.permutation(blocks), pages, int(pages.max()), n)
    cumseq = np.concatenate([[0], np.cumsum(q)])
    T = int(cumseq[-1])
    seq = np.repeat(np.arange(n), q)
    pos = ctx[seq] - q[seq] + np.arange(T) - cumseq[seq]
    slots = table[seq, pos // bs].astype(np.int64) * bs + pos % bs

    def normal(*shape):
        return torch.empty(*shape, dtype=dt, device=DEV).normal_(0.0, 1.0, generator=gen)

    rows = int(ctx.max())
    ang = np.arange(rows)[:, None] * np.power(10000.0, -2.0 * np.arange(hs // 2)[None, :] / hs)
    s = {"case": c, "query": normal(T, H * 2 * hs), "key": normal(T, kv * 2 * hs), "value": normal(T, kv * vhs),
         "kc": normal(blocks, bs, kv, 2, hs), "vc": normal(blocks, bs, kv, vhs), "cos": _dev(np.cos(ang), dt),
         "sin": _dev(np.sin(ang), dt),
         "lam": torch.empty(4, hs, device=DEV).normal_(0.0, 0.1, generator=gen),
         "norm": (1.0 + 0.1 * torch.empty(vhs, device=DEV).normal_(0.0, 1.0, generator=gen)).to(dt),
         "cumseq": _dev(cumseq), "past": _dev(ctx - q), "table": _dev(table), "slots": _dev(slots),
         "longest": rows, "tokens": T}
    if own:
        from paged_latent_attention_cache_gb300.api import DifferentialAttention
        s["op"] = DifferentialAttention(
            dtype=dt, num_heads=H, kv_num_heads=kv, head_size=hs, v_head_size=vhs, rotary_dim=hs, cos_rows=rows,
            block_size=bs, num_blocks=blocks, max_blocks_per_seq=table.shape[1], local_window_size=c["window"],
            lambda_init=_lambda_init(c), max_seqs=n, max_tokens=T, own_slots=True)
    return s


def _lambda_init(c):
    return 0.8 - 0.6 * math.exp(-0.3 * c["depth"])


# -------------------------------------------------------------------------------------------- runs

def run(state):
    return {"copy": _copy, "fork": _fork, "compact": _compact, "step": _step, "attend": _attend}[state["case"]["op"]](state)


def _bits(caches):
    return [t.view(torch.int16) for t in caches]


def _copy(s):
    if own:
        s["pool"].copy(s["src"], s["dst"], s["rows"])
    else:
        _copy_rows(s["caches"], s["src"], s["dst"], s["rows"])
    return {"caches": _bits(s["caches"])}


def _copy_rows(caches, src, dst, rows):
    src, dst = src.long(), dst.long()
    if rows is None:
        return [t.index_copy_(1, dst, t[:, src]) for t in caches]
    keep = (torch.arange(caches[0].shape[2], device=DEV)[None, :] < rows[:, None])[None, :, :, None]
    return [t.index_copy_(1, dst, torch.where(keep, t[:, src], t[:, dst])) for t in caches]


def _plain_free(s, rows):
    rows = rows.long()
    gone = s["table"][rows].flatten()
    s["ref"].index_add_(0, gone.clamp(min=0).long(), -(gone >= 0).int())
    s["table"].index_fill_(0, rows, -1)
    s["past"].index_fill_(0, rows, 0)


def _fork(s):
    """A beam step: the old beams are freed, then every prompt is forked anew."""
    if own:
        s["pool"].free(s["children"])
        s["pool"].fork(s["parents"], s["children"])
    else:
        _plain_free(s, s["children"])
        _plain_fork(s, s["parents"].long(), s["children"].long(), s["case"]["bs"])
    return {"caches": _bits(s["caches"]), "table": s["table"], "past": s["past"], "ref": s["ref"]}


def _plain_fork(s, parents, children, bs):
    table, past, ref = s["table"], s["past"], s["ref"]
    ctx, prow = past[parents], table[parents]
    full, tail = (ctx // bs)[:, None], ctx % bs
    need = tail > 0
    free = torch.argsort((ref != 0).int(), stable=True)  # the free pages, lowest first
    new = torch.where(need, free[(torch.cumsum(need, 0) - 1).clamp(min=0)].int(), -1)
    j = torch.arange(table.shape[1], device=DEV, dtype=torch.int32)[None, :]
    shared = (j < full) & (prow >= 0)
    ref.index_add_(0, prow.clamp(min=0).flatten().long(), shared.flatten().int())
    ref.index_add_(0, new.clamp(min=0).long(), need.int())
    table[children] = torch.where(shared, prow, torch.where((j == full) & need[:, None], new[:, None], -1))
    past[children] = ctx
    old = torch.gather(prow, 1, full.clamp(max=table.shape[1] - 1).long())[:, 0]
    old = torch.where(need, old, prow[:, 0])  # a full last page: nothing to copy, a page onto itself
    _copy_rows(s["caches"], old, torch.where(need, new, old), torch.where(need, tail, 0))


def _compact(s):
    s["table"].copy_(s["table0"])  # the scattered pool again (the rows of moved pages are still there)
    s["ref"].copy_(s["ref0"])
    if own:
        s["pool"].compact()
    else:
        table, ref = s["table"], s["ref"]
        ids = torch.arange(ref.numel(), device=DEV)
        live = ref > 0
        count = live.sum()
        dst, src = (~live & (ids < count)).nonzero()[:, 0], (live & (ids >= count)).nonzero()[:, 0]
        _copy_rows(s["caches"], src, dst, None)
        to = ids.int().index_copy_(0, src, dst.int())
        table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -1))
        ref.index_copy_(0, dst, ref[src])
        ref.index_fill_(0, src, 0)
    return {"caches": _bits(s["caches"]), "table": s["table"], "ref": s["ref"]}


def _step(s):
    """One step of continuous batching: the rows that ended are freed and taken by new prompts, the
    others go on by a token; every row gets the pages and the tokens their cache slots."""
    if own:
        s["pool"].free(s["ended"])
        s["pool"].reserve(s["cumseq"], s["slots"])
    else:
        _plain_free(s, s["ended"])
        _plain_reserve(s, s["case"]["bs"])
    return {"table": s["table"], "past": s["past"], "ref": s["ref"], "slots": s["slots"]}


def _plain_reserve(s, bs):
    table, past, ref, cumseq = s["table"], s["past"], s["ref"], s["cumseq"]
    q = cumseq[1:] - cumseq[:-1]
    want = ((past + q + bs - 1) // bs)[:, None]
    j = torch.arange(table.shape[1], device=DEV, dtype=torch.int32)[None, :]
    lack = (j < want) & (table < 0) & (q > 0)[:, None]
    fits = torch.cumsum(lack.sum(1), 0) <= (ref == 0).sum()
    lack &= fits[:, None]
    free = torch.argsort((ref != 0).int(), stable=True)
    rank = (torch.cumsum(lack.flatten(), 0) - 1).clamp(min=0, max=ref.numel() - 1)
    table.copy_(torch.where(lack, free[rank].int().view_as(table), table))
    ref.index_add_(0, table.clamp(min=0).flatten().long(), lack.flatten().int())
    seq = torch.repeat_interleave(torch.arange(q.numel(), device=DEV), q, output_size=s["tokens"])
    pos = past[seq] + torch.arange(s["tokens"], device=DEV, dtype=torch.int32) - cumseq[seq]
    page = table[seq, (pos // bs).long()]
    s["slots"].copy_(torch.where(fits[seq] & (page >= 0), page * bs + pos % bs, -1))


def _attend(s):
    if own:
        c = s["case"]
        out = s["op"].forward(s["query"], s["key"], s["value"], s["kc"], s["vc"], s["cos"], s["sin"], s["lam"], s["norm"],
                              s["cumseq"], s["past"], s["table"], s["slots"],
                              num_decode_seqs=c["seqs"] if c["q"] == 1 else 0)
    else:
        out = _plain_attend(s)
    return {"out": out, "kc": s["kc"], "vc": s["vc"]}


def _rope(x, cos, sin):
    """Half-split rotation of the last axis; cos and sin broadcast over the heads."""
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_attend(s):
    c = s["case"]
    H, kv, hs, vhs, bs, n, Q = c["heads"], c["kv"], c["hs"], c["vhs"], c["bs"], c["seqs"], c["q"]
    dt, T, L = s["query"].dtype, s["tokens"], s["longest"]
    G = H // kv
    past = s["past"].long()
    pos = past[:, None] + torch.arange(Q, device=DEV)[None, :]  # [n, Q]: every sequence has Q new tokens
    cos, sin = (t.float()[pos.flatten()][:, None, None, :] for t in (s["cos"], s["sin"]))
    k = _rope(s["key"].float().view(T, kv, 2, hs), cos, sin).to(dt)
    s["kc"].view(-1, kv, 2, hs).index_copy_(0, s["slots"].long(), k)
    s["vc"].view(-1, kv, vhs).index_copy_(0, s["slots"].long(), s["value"].view(T, kv, vhs))
    q = _rope(s["query"].float().view(T, H, 2, hs), cos, sin).view(n, Q, kv, G, 2, hs)
    j = torch.arange(L, device=DEV)
    row = s["table"].long()[:, j // bs].clamp(min=0) * bs + j % bs  # [n, L]
    K = s["kc"].view(-1, kv, 2, hs)[row].float()  # [n, L, kv, 2, hs]
    V = s["vc"].view(-1, kv, vhs)[row].float()
    q = q.permute(0, 2, 4, 3, 1, 5).reshape(n, kv, 2, G * Q, hs) * (1.0 / math.sqrt(hs))
    x = (q @ K.permute(0, 2, 3, 4, 1)).view(n, kv, 2, G, Q, L)
    seen = j[None, None, :] <= pos[:, :, None]
    if c["window"] >= 0:
        seen = seen & (pos[:, :, None] - j[None, None, :] <= c["window"])
    x.masked_fill_(~seen[:, None, None, None], -math.inf)
    x -= x.amax(-1, keepdim=True)
    x.exp_()
    x /= x.sum(-1, keepdim=True)
    v = s["lam"]
    lam = torch.exp((v[0] * v[1]).sum()) - torch.exp((v[2] * v[3]).sum()) + _lambda_init(c)
    d = x[:, :, 0] - lam * x[:, :, 1]
    o = d.view(n, kv, G * Q, L) @ V.permute(0, 2, 1, 3)  # [n, kv, G*Q, vhs]
    o = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + 1e-5) * s["norm"].float() * (1.0 - _lambda_init(c))
    return o.view(n, kv, G, Q, vhs).permute(0, 3, 1, 2, 4).reshape(T, H * vhs).to(dt)


# -------------------------------------------------------------------------------- work and exactness

def _mean_context(c):
    n = c["seqs"] if "seqs" in c else c["parents"]
    return float(np.linspace(c["hi"], c["lo"], n + 1)[:n].mean())


def work(case):
    """Bytes and operations of one pass: what is read once and written once. Lengths that the inputs
    draw at random count with their mean."""
    c = case
    if c["op"] == "attend":
        n, q, H, kv, hs, vhs = c["seqs"], c["q"], c["heads"], c["kv"], c["hs"], c["vhs"]
        ctx = _mean_context(c)
        T = n * q
        past = ctx - q
        if c["window"] < 0:
            pairs, rows = n * (q * past + q * (q + 1) / 2), n * ctx
        else:
            w = c["window"] + 1
            a = max(0.0, min(float(q), w - past))  # new tokens that still see everything before them
            pairs = n * (a * past + a * (a + 1) / 2 + (q - a) * w)
            rows = n * min(ctx, w + q - 1)
        row = kv * (2 * hs + vhs)
        nbytes = 2 * (rows * row + T * H * (2 * hs + vhs) + 2 * T * row + 2 * T * hs) + 4 * n * ctx / c["bs"]
        return {"bytes": nbytes, "flops": pairs * H * 2 * 2 * (hs + vhs)}
    if c["op"] == "step":
        free = c["ended"] * (c["hi"] / 2 + c["prompt"]) / c["bs"]
        tokens = c["seqs"] - c["ended"] + c["ended"] * c["prompt"]
        return {"bytes": 4 * (4 * free + tokens + 4 * c["seqs"] + c["blocks"]), "flops": tokens}
    row = c["layers"] * (c["width"] + c["vwidth"]) * 2
    if c["op"] == "copy":
        return {"bytes": 2 * row * c["n"] * (0.5 * (c["bs"] + 1) if c["rows"] else c["bs"]), "flops": 0}
    if c["op"] == "fork":
        kids = c["parents"] * c["beams"]
        table = kids * _mean_context(c) / c["bs"]
        return {"bytes": 2 * row * kids * 0.5 * (c["bs"] - 1) + 4 * 6 * table, "flops": table}
    moved = c["blocks"] * c["live"] * (1.0 - c["live"])
    return {"bytes": 2 * row * moved * c["bs"] + 4 * (2 * c["blocks"] + 3 * c["blocks"] * c["live"]), "flops": c["blocks"]}


def exact(case, seed):
    """Differential attention sequence by sequence and head by head in 64 bits. The page operators
    give whole numbers and copies."""
    c = case
    if c["op"] != "attend":
        return None
    if c["seqs"] * c["heads"] * c["q"] * c["hi"] > 3e9:
        return None
    s = prepare(case, seed)
    H, kv, hs, vhs, bs = c["heads"], c["kv"], c["hs"], c["vhs"], c["bs"]
    past, cum, table = s["past"].tolist(), s["cumseq"].tolist(), s["table"].tolist()
    key, value, query = (s[k].double() for k in ("key", "value", "query"))
    kc, vc = s["kc"].clone(), s["vc"].clone()
    out = torch.empty(s["tokens"], H, vhs, dtype=torch.float64, device=DEV)
    lv = s["lam"].double()
    lam = math.exp(float(lv[0] @ lv[1])) - math.exp(float(lv[2] @ lv[3])) + _lambda_init(c)
    half = hs // 2

    def turn(x, p):  # x [tokens, hs] at positions p
        co, si = s["cos"][p].double(), s["sin"][p].double()
        y = torch.empty_like(x)
        y[:, :half] = x[:, :half] * co - x[:, half:] * si
        y[:, half:] = x[:, half:] * co + x[:, :half] * si
        return y

    for b in range(c["seqs"]):
        t0, t1, p0 = cum[b], cum[b + 1], past[b]
        p = torch.arange(p0, p0 + t1 - t0, device=DEV)
        ctx = p0 + t1 - t0
        pages = torch.tensor(table[b][:-(-ctx // bs)], device=DEV)
        slot = (pages[:, None] * bs + torch.arange(bs, device=DEV)[None, :]).flatten()[:ctx]
        j = torch.arange(ctx, device=DEV)
        hidden = j[None, :] > p[:, None]
        if c["window"] >= 0:
            hidden = hidden | (p[:, None] - j[None, :] > c["window"])
        for g in range(kv):
            for i in range(2):
                at = (g * 2 + i) * hs
                kc.view(-1, kv, 2, hs)[slot[p0:], g, i] = turn(key[t0:t1, at:at + hs], p).to(kc.dtype)
            vc.view(-1, kv, vhs)[slot[p0:], g] = s["value"][t0:t1, g * vhs:(g + 1) * vhs]
            V = vc.view(-1, kv, vhs)[slot, g].double()
            for h in range(g * (H // kv), (g + 1) * (H // kv)):
                maps = []
                for i in range(2):
                    at = (h * 2 + i) * hs
                    K = kc.view(-1, kv, 2, hs)[slot, g, i].double()
                    x = turn(query[t0:t1, at:at + hs], p) @ K.T / math.sqrt(hs)
                    x[hidden] = -math.inf
                    maps.append(torch.softmax(x, -1) @ V)
                o = maps[0] - lam * maps[1]
                o = o / torch.sqrt((o ** 2).mean(-1, keepdim=True) + 1e-5)
                out[t0:t1, h] = o * s["norm"].double() * (1.0 - _lambda_init(c))
    return {"out": out.view(s["tokens"], H * vhs), "kc": None, "vc": None}
