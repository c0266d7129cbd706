"""Every kernel of the library is launched with programmatic dependent launch, so it may start while the
kernel before it still runs, and earlier writes on the stream are visible to it only behind its own
griddepcontrol.wait. Read off the sources (no GPU): each kernel waits once, on every path, before
its first access to global memory."""
import glob
import os
import re

import pytest

import bit_quantization_aware_blockwise_b200 as q

CSRC = os.path.join(os.path.dirname(os.path.abspath(q.__file__)), "csrc")


def without_comments(text):
    text = re.sub(r"//[^\n]*", "", text)
    return re.sub(r"/\*.*?\*/", "", text, flags=re.S)


def kernels():
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = without_comments(open(path).read())
        for m in re.finditer(r"__global__\s+void\s+(?:__\w+__\([^;{]*?\)\s+)*(\w+)\(", text):
            start = at = text.index("{", m.end())
            depth = 0
            while True:
                depth += {"{": 1, "}": -1}.get(text[at], 0)
                at += 1
                if depth == 0:
                    break
            found.append((os.path.basename(path), m.group(1), text[start + 1:at - 1]))
    return found


KERNELS = kernels()
READS = re.compile(r"__ldg|__ldcs|__ldcv|copy_async|copy16_async|fetch_x\(|stage_x<|tma_load|tma_store|cp\.async\.(ca|cg)|ld\.global|"
                   r"atomic")


def test_the_kernels_are_found():
    names = {k for _, k, _ in KERNELS}
    assert {"lowbit_kernel", "stage_kernel", "weight_grad_kernel", "weight_grad_finish_kernel", "restore_codes_kernel",
            "gated_pair_kernel", "gated_zero_kernel", "gated_bwd_kernel", "zero_fill_kernel"} <= names
    total = sum(without_comments(open(p).read()).count("__global__") for p in glob.glob(os.path.join(CSRC, "*.cu")))
    assert len(KERNELS) == total


@pytest.mark.parametrize("file,kernel,body", KERNELS, ids=[k for _, k, _ in KERNELS])
def test_waits_on_every_path_before_it_reads(file, kernel, body):
    assert body.count("pdl_wait()") == 1
    before = body[:body.index("pdl_wait()")]
    assert before.count("{") == before.count("}"), "the wait is inside a block"
    assert re.search(r"[;{}]\s*$", before) or not before.strip(), "the wait is conditional"
    assert not READS.search(before)
