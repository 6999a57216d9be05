"""Rules of the kernels that no result shows, checked on their sources: what breaks them
breaks a run only now and then."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "fp8_moe_routed_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def code(path):
    with open(path) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_barriers_of_the_peer_cta_are_waited_for_at_cluster_scope(path):
    """A barrier that is addressed through mapa (threads or copies of the peer CTA arrive on
    it) is waited for and tested with an acquire at cluster scope."""
    text = code(path)
    shared = set(re.findall(r"mapa_shared\(smem_u32\(&s\.(\w+)", text))
    for wait, name in re.findall(r"(mbar_(?:try_)?(?:wait|test)\w*)\(&s\.(\w+)", text):
        assert name not in shared or wait.endswith("_cluster"), (wait, name)


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_shared_byte_arrays_are_aligned_for_the_words_read_from_them(path):
    """Arrays of a kernel's own (dynamic shared memory is aligned by where it starts)."""
    text = code(path)
    for name in re.findall(r"(?<!extern )__shared__\s+uint8_t\s+(\w+)\s*\[", text):
        assert not re.search(r"reinterpret_cast<[^>]*\*>\(\s*&?%s\b" % name, text), name


def test_the_norms_leave_no_copy_in_flight_behind_a_failed_wait():
    """A wait for a row that runs out ends the filling of the ring, but not the waits for the
    rows that were on their way: a CTA gives up on as many as it has stages."""
    text = code(os.path.join(CSRC, "norm.cu"))
    assert re.search(r"kAllLost = kOneLost \* kMaxStages;", text)
    assert re.search(r"if \(state < kAllLost && !mbar_wait\(.*?\)\) state \+= kOneLost;", text)
    kernels = [k for k in re.split(r"__global__", text)[1:] if "ring.fill" in k]
    assert len(kernels) == 2
    for k in kernels:
        body = k[k.index("for (uint32_t row = row0"):]
        assert body.count("wait_row(ring, stage, state);") == 1 and "mbar_wait" not in body
        fills = re.findall(r"if \(([^;{]*?)\)\s*ring\.fill", body)
        assert len(fills) == body.count("ring.fill") > 0
        assert all("state < kOneLost" in f for f in fills), fills


def test_no_norm_variant_is_built_that_no_row_reaches():
    """f32 rows hold at most 8192 values, which 512 threads take: the variants of 1024 threads
    are bf16's alone. By the compiler's report of the build at hand."""
    report = os.path.join(os.path.dirname(CSRC), "_build", "norm.cu.ptxas.txt")
    if not os.path.exists(report):
        pytest.skip("not built here")
    with open(report) as f:
        built = set(re.findall(r"norm_(?:fwd|bwd)_kernelI(\w+?)Li(\d+)E", f.read()))
    assert built == {("13__nv_bfloat16", "512"), ("13__nv_bfloat16", "1024"), ("f", "512")}
