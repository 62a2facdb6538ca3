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
