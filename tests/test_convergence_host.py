"""Instructions that a whole warp has to execute together (tensor-memory loads and
allocation, cluster barriers: ".aligned") in the dense products' kernels stand behind a
meeting of the warp wherever its lanes may have parted.  A warp that arrives in parts may
never return, so this is read from the sources, not run."""
import glob
import os
import re

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "latent_mixture_experts_gb300", "csrc")
FILES = [*sorted(glob.glob(os.path.join(CSRC, "ffn_*.cu"))), os.path.join(CSRC, "dense_gemm.cu")]
MEET = re.compile(r"__syncwarp\(|__syncthreads\(|cluster_wait\(|cluster_sync\(|named_sync\(")


def _code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _body(text, at):
    """The braces' content that begins behind `at`."""
    at = text.index("{", at)
    depth, i = 0, at
    while True:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
        if depth == 0:
            return text[at + 1:i - 1]


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_loads_from_tensor_memory_follow_a_meeting(path):
    text = _code(path)
    for m in re.finditer(r"for \(int c0? = [^{]*\{", text):
        body = _body(text, m.start())
        if not re.search(r"tmem_ld(16|32)\(", body):
            continue
        parts = [x for x in re.findall(r"if \(([^\n]*)", body) if "break" not in x and "constexpr" not in x]
        if parts:      # lanes may part: the last statement brings them together
            last = body.strip().rstrip("}").strip().splitlines()[-1].strip()
            assert re.match(r"__syncwarp\(\);|store_rows\(", last), body


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_barriers_follow_a_meeting(path):
    lines = [x.strip() for x in _code(path).splitlines() if x.strip()]
    for i, x in enumerate(lines):
        if not re.search(r"\b(cluster_arrive|cluster_sync|tmem_alloc|tmem_alloc_pair)\(", x):
            continue
        assert any(MEET.search(y) for y in lines[max(0, i - 6):i]), lines[max(0, i - 6):i + 1]
