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
