"""What the memory model asks of the kernels' sources, where a GPU run does not show the
difference."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "latent_mixture_experts_sigmoid_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def test_arrivals_in_another_cta_name_their_scope():
    # an arrive's scope is the CTA unless it says otherwise: too little for a barrier that may
    # be another CTA's
    found = 0
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        for m in re.finditer(r'"(mbarrier\.arrive[^ "]*\.shared::cluster[^ "]*)', open(path).read()):
            found += 1
            assert ".cluster.shared::cluster" in m[1], (path, m[1])
    assert found >= 2


def test_data_handed_to_the_other_cta_is_released_and_acquired():
    # (weights' gradient: the zeros behind an expert's last row are read by the leader's MMAs)
    ptx, grouped = source("tc_ptx.cuh"), source("grouped.cu")
    body = re.search(r"void mbar_arrive_cluster_data\(.*?\n}", ptx, re.S)[0]
    assert "mbarrier.arrive.release.cluster.shared::cluster" in body
    assert "parity.acquire.cluster" in re.search(r"void mbar_acquire_cluster\(.*?\n}", ptx, re.S)[0]
    mma = grouped[grouped.index("MMA issuer of the pair"):grouped.index("warp == 2")]
    # behind the wait for the block, ahead of its MMAs
    assert mma.index("kFull + s), ph, abort_flag") < mma.index("mbar_acquire_cluster(") < mma.index("mma_pair(")
