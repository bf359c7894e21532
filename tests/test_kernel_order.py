"""Waits in the kernels that no run can show to be missing: a run without them
nearly always passes. They are looked for in the source."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_latent_attention_cache_gb300", "csrc")


def _source(name):
    src = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", src)


def _kernels(src):
    """name -> body of every __global__ function."""
    found = {}
    for m in re.finditer(r"__global__\s+void\b", src):
        head = src[m.end():src.index("{", m.end())]
        head = re.sub(r"__\w+__\s*\(([^()]|\([^()]*\))*\)", "", head)
        name = re.search(r"(\w+)\s*\(", head).group(1)
        at = src.index("{", m.end())
        depth, end = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(src[end], 0)
            end += 1
            if depth == 0:
                break
        found[name] = src[at:end]
    return found


def test_cluster_has_started_before_its_shared_memory_is_written():
    """warp_prefix stores into the shared memory of every CTA of the cluster:
    each kernel passes a barrier of the cluster before its first one, and one
    that splits it arrives before anything can wait."""
    users = {k: b for k, b in _kernels(_source("pa_pages.cu")).items() if "warp_prefix<" in b}
    assert set(users) == {"fork_plan_kernel", "reserve_kernel", "compact_plan_kernel"}
    for name, body in users.items():
        first = body.index("warp_prefix<")
        at = [body.find(w) for w in ("cl.sync()", "cluster_started()")]
        assert any(0 <= a < first for a in at), name
        assert body.count("cluster_start()") == body.count("cluster_started()"), name
        if "cluster_start()" in body:
            assert body.index("cluster_start()") < body.index("chain()") < body.index("cluster_started()"), name


def _first_wrong_wait(n, bufs, last_wait):
    """The order of one CTA of diff_prefill_kernel, values as late as can be:
    the scores of tile k are there once the products issued before them are,
    and PV of tile j waits for its values. Returns the tile at which a wait of
    the softmax for PV passes although that PV is not done, else None.
    ``pv_done`` has two barriers; a wait for a phase's parity passes when the
    phase in progress has the other one."""
    done = -1  # the last PV done
    phases = [0, 0]

    def finish(upto):
        nonlocal done
        while done < upto:
            done += 1
            phases[done & 1] += 1

    def passes(k):  # a wait for PV of tile k
        return phases[k & 1] & 1 != (k >> 1) & 1

    for k in range(n):
        finish(k - bufs)  # QK^T of tile k was issued behind PV of tile k - bufs
        if k > 0 and passes(k - 1) and done < k - 1:
            return k  # (O is scaled in place behind this one)
    if last_wait == "pv_done" and passes(n - 1) and done < n - 1:
        return n
    return None


def test_prefill_waits_for_all_products():
    """A wait for the last tile's phase of pv_done can return at once with three
    buffers, whatever the number of tiles above two; the waits inside the tiles
    cannot. So the kernel's last wait is for a barrier with a single phase,
    behind every product."""
    for n in range(1, 40):
        assert _first_wrong_wait(n, 2, "pv_done") is None
        assert _first_wrong_wait(n, 3, "pv_done") == (n if n >= 3 else None)
        assert _first_wrong_wait(n, 2, "drain") is None and _first_wrong_wait(n, 3, "drain") is None
    body = _kernels(_source("pa_diff_prefill.cu"))["diff_prefill_kernel"]
    softmax = body[body.index("auto rescale_o"):body.index("coef = lt")]
    tiles, end = softmax[:softmax.index("grid_dep_launch()")], softmax[softmax.index("grid_dep_launch()"):]
    assert tiles.count("pv_done") == 1 and "pv_done" not in end
    assert "wait_bar(smem_u32(&bars->drain), 0," in end
    assert body.count("tc_commit(smem_u32(&bars->drain))") == 1


def test_prefill_stores_to_tensor_memory_in_order():
    """The probabilities of a tile may be stored twice to the same columns:
    tcgen05.st is asynchronous, so the first stores are waited for between."""
    body = _kernels(_source("pa_diff_prefill.cu"))["diff_prefill_kernel"]
    tile = body[body.index("bool again"):body.index("arrive_warp(p_full")]
    first, second = [m.start() for m in re.finditer(r"\bexps\(\)", tile)]
    assert "tmem_wait_st()" in tile[first:second]


def test_decode_leaves_no_copy_in_flight():
    """Every way out of the loop over a CTA's part that leaves tiles unread is
    followed by a wait for the copies that were started."""
    body = _kernels(_source("pa_diff_decode.cu"))["diff_decode_kernel"]
    assert re.search(r"if \(seg <= 0[^;]*\) break;", body)  # tiles left: at < count
    end = body[body.index("s_cur = cur;"):]
    wait = end[:end.index("drain_wait")]
    assert "s_abort || at < count" in wait
