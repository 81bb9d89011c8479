"""How the CTAs of a pair hand shared and tensor memory to each other (CPU only, on the sources).

A thread that waits on a barrier sees what was done before an arrival there only if the arrival is a
release and the wait an acquire, both at a scope that holds both threads: for two CTAs of a cluster,
cluster scope.  Copies count as a release at cluster scope by their own completion on the barrier."""
import pathlib
import re

CSRC = pathlib.Path(__file__).resolve().parents[1] / "expert_cached_sparse_b200" / "csrc"


def code(name):
    s = re.sub(r"/\*.*?\*/", "", (CSRC / name).read_text(), flags=re.S)
    return re.sub(r"//[^\n]*", "", s)


def test_arrivals_in_another_cta_are_releases_at_cluster_scope():
    s = code("tc.cuh")
    remote = re.findall(r'"(mbarrier\.arrive[\w.:]*shared::cluster[\w.:]*)', s)
    assert remote
    for op in remote:   # an arrival that only announces copies has nothing of its own to publish
        assert ".release.cluster." in op or ".expect_tx.relaxed.cluster." in op, op


def test_a_pairs_waits_acquire_at_cluster_scope():
    s = code("tc.cuh")
    assert "mbarrier.try_wait.parity.acquire.cluster.shared::cta" in s
    g = code("grouped_gemm.cu")
    # every wait that a pair of CTAs reaches names the pair; `ready` is DW's, whose CTAs stand alone
    for m in re.finditer(r"mbar_(?:wait|wait_warp|drain)(<[^>]*>)?\(smem_u32\(&(\w+)", g):
        assert m.group(1) in ("<CG>", "<2>") or m.group(2) == "full" and "MODE == DW" in g[: m.start()][-700:], m.group(0)
    assert re.search(r"mbar_wait<CG>\(bar,", g) and re.search(r"copy_loop<STAGE, CG>\(full0,", g)
