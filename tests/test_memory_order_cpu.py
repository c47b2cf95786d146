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
    assert found >= 1


def test_no_thread_writes_what_the_other_cta_s_tensor_cores_read():
    # (grouped products: every operand comes by TMA, whose bytes count on the leader's barrier; a CTA's
    # threads write their epilogue's boxes alone.  Otherwise a release and an acquire of cluster scope
    # have to stand between the writes and the MMAs.)
    grouped = source("grouped.cu")
    roles = grouped[grouped.index("TMA producer ---"):grouped.index("epilogue ---")]
    assert "mma_pair(" in roles and "reinterpret_cast<uint4*>" not in roles
    if "mbar_arrive_cluster_data" in grouped:
        assert "mbarrier.arrive.release.cluster" in source("tc_ptx.cuh") and "acquire.cluster" in source("tc_ptx.cuh")


def test_in_place_operands_are_not_read_as_constant():
    # ld.global.nc and __restrict__ say that nobody writes the memory while the kernel runs; SituGLU's
    # gradient may be written over its input, the norm's outputs over its inputs
    situ = source("situ.cu")
    kernel = re.search(r"situ_backward_kernel\(.*?\n}", situ, re.S)[0]
    assert re.match(r"situ_backward_kernel\(const uint16_t\* in,", kernel), kernel[:80]
    loads = re.findall(r"(\w+)\(reinterpret_cast<const uint4\*>\(in \+", kernel)
    assert len(loads) == 2
    for name in loads:
        assert ".nc" not in re.search(r"uint4 " + name + r"\(.*?\n}", situ, re.S)[0], name
    norm = source("norm.cu")
    assert ".nc" not in norm and "__ldg" not in norm


def test_tensor_maps_have_the_documented_form():
    # each stride is the one before times its extent (a map with two equal strides counts rows twice
    # and covers memory that its matrix does not have), and no copy of token rows begins ahead of them
    grouped = source("grouped.cu")
    strides = re.findall(r"cuuint64_t strides\[\d\] = \{(.*?)\};", grouped)
    assert strides == ["(cuuint64_t)cols * size, (cuuint64_t)cols * size * (cuuint64_t)rows"]
    producer = grouped[grouped.index("TMA producer ---"):grouped.index("MMA issuer of the pair")]
    rows = set(re.findall(r"box\(&maps\.\S+, &maps\.\S+, \w+, ([^)]*)\)", producer))
    assert rows == {"row0", "row0 + r", "beyond"} and "const int row0 = x.row0 + k, beyond = (int)p.R;" in producer
