"""Rules that every kernel source keeps, checked on the sources themselves: they
concern faults that no run on a GPU may be made to show."""
import glob
import os
import re

from bmm_reducescatter_alltoall_gb300._build import CSRC, code_text


def sources():
    """Code text of each kernel source and header, adjacent string literals joined."""
    files = sorted(glob.glob(os.path.join(CSRC, "*.cu*")))
    assert len(files) > 15
    for path in files:
        with open(path, "rb") as f:
            yield os.path.basename(path), re.sub(r'"\s*"', "", code_text(f.read()).decode())


def test_no_bulk_copy_is_multicast():
    """The library also runs as one rank of several: its copies write the issuing CTA's shared
    memory alone (a commit's arrivals are no copies)."""
    for name, text in sources():
        assert not re.search(r"cp\.(async|reduce)[\w.:]*multicast", text), name


# Kernels that begin before the one ahead of them in the stream has ended, and what they share.
OVERLAPPED = {"grouped_aux.cu", "grouped_split.cu", "grouped_tc.cu", "moe_permute.cu", "moe_route.cu",
              "mx_quant.cu", "mx_tc.cu"}
SHARED = {"grouped.cuh", "launch.cuh", "mx.cuh", "walk.cuh", "moe_internal.h"}


def test_overlapped_kernels_read_with_loads_that_see_writes():
    """Their inputs may be written while they already run: no load for constant data."""
    seen = set()
    for name, text in sources():
        if name.endswith(".cu"):
            assert (name in OVERLAPPED) == ("ProgrammaticStreamSerialization" in text or
                                            "launch_overlapped" in text), name
        if name in OVERLAPPED | SHARED:
            seen.add(name)
            assert not re.search(r"__ldg\b|__restrict__|__restrict\b|ld\.global[\w.]*\.nc\b", text), name
    assert seen >= OVERLAPPED


def test_cluster_barriers_follow_a_barrier_of_the_warp():
    """Their instructions are for whole warps (.aligned): the lanes have to be together again."""
    found = 0
    for name, text in sources():
        for m in re.finditer(r"cluster_sync\(\);", text):
            found += 1
            assert re.search(r"__sync(threads|warp)\(\);\s*(}\s*)?(if \(CG == 2\) )?$",
                             text[:m.start()]), (name, text[m.start() - 120:m.end()])
    assert found > 8
