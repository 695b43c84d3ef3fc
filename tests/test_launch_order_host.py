"""Source rule of the kernels launched with programmatic stream serialisation:
no block leaves before it has waited for the kernel before it, since whatever
follows in the stream is ordered behind the launched kernel alone."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "compressed_sparse_attention_11_b200", "csrc")


def waiting_kernels():
    """(file, kernel, body) of every kernel that calls pdl_wait(), comments taken out."""
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for chunk in text.split("__global__")[1:]:
            name = re.search(r"(\w+)\s*\(", re.sub(r"__launch_bounds__\s*\([^)]*\)", "", chunk)).group(1)
            body = re.split(r"\n}\n", chunk)[0]      # a kernel ends at the first brace in column 0
            if "pdl_wait();" in body:
                found.append((os.path.basename(path), name, body))
    return found


def test_the_kernels_are_found():
    names = {k[1] for k in waiting_kernels()}
    assert {"kv4_decode_kernel", "kv4_combine_kernel", "decode_combine_kernel", "append_emit_kernel",
            "decode_topk_hist_kernel"} <= names


@pytest.mark.parametrize("file,name,body", waiting_kernels(), ids=[k[1] for k in waiting_kernels()])
def test_no_exit_before_the_wait(file, name, body):
    assert not re.search(r"\breturn\s*;", body[:body.index("pdl_wait();")]), f"{file}: {name}"
    trigger = body.find("pdl_trigger();")
    assert trigger < 0 or body.index("pdl_wait();") < trigger, f"{file}: {name}"
