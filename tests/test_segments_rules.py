"""Rules of the segmented products' sources that a run on one GPU cannot show,
checked on the CPU by reading them."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "dense_fp32_gemm_major_gb300", "csrc")


def sources():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".h")):
            with open(os.path.join(CSRC, name)) as f:
                text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
            yield name, re.sub(r"//[^\n]*", "", text)


def once_bodies(text):
    """The bodies of the lambdas given to call_once."""
    for m in re.finditer(r"\bcall_once\s*\([^{]*\{", text):
        depth, i = 1, m.end()
        while depth and i < len(text):
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield text[m.end():i]


# What the runtime keeps for each device: done once a process, it is missing on
# every GPU but the first one used.
PER_DEVICE = re.compile(r"cudaFuncSetAttribute|cudaFuncGetAttributes|cudaMemPool\w*|cudaMemcpyToSymbol")


def test_what_a_device_keeps_is_not_set_once_a_process():
    seen = 0
    for name, text in sources():
        for body in once_bodies(text):
            seen += 1
            assert not PER_DEVICE.search(body), f"{name}: {PER_DEVICE.search(body).group(0)}"
    assert seen >= 2  # the driver's entry points
    assert list(once_bodies("std::call_once(o, [&] { if (a) { b(); } c(); }); d();")) \
        == [" if (a) { b(); } c(); }"]


def arrivals(text):
    """(address space, qualifiers) of every mbarrier.arrive in the text's PTX."""
    for m in re.finditer(r"mbarrier\.arrive((?:\.[a-z_]+)*)\.(shared::\w+)\.b64", text):
        yield m.group(2), m.group(1).split(".")[1:]


def test_arrivals_at_another_cta_have_its_scope():
    # Without a scope an arrival is a release at CTA scope, which a thread of
    # another CTA cannot acquire: what it announces would be unordered.
    remote = 0
    for name, text in sources():
        for space, qualifiers in arrivals(text):
            if space == "shared::cluster":
                remote += 1
                assert "cluster" in qualifiers, f"{name}: {qualifiers}"
    assert remote >= 2
    assert list(arrivals('"mbarrier.arrive.shared::cluster.b64 _, [%0];"')) == [("shared::cluster", [])]
    assert list(arrivals("mbarrier.arrive.release.cluster.shared::cluster.b64")) == [
        ("shared::cluster", ["release", "cluster"])]


def test_the_dense_kernels_recorded_traffic_is_of_their_sources():
    # DRAM bytes are on record by the hash of a kernel's sources: what only the
    # segmented products need is no part of them
    import bench

    for kernel, mode in (("tc_pair_tma_3xtf32", "exact"), ("tc_pair_tma_tf32", "tf32"),
                         ("simt_gemm", "exact_simt")):
        assert bench.traffic_lookup(kernel, "c4", mode)[0] is not None, kernel
