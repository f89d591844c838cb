"""CPU: exchanges among a wave's lanes through LDS stay in the compiled code.

The gradient kernel finds an expert named twice by writing a tag to the
expert's place and reading it back: another lane may have written there. To the
compiler, a load after a store to the same address is the value stored, unless
the source says otherwise. Here the kernel is compiled for rows of at most 16
entries, where nothing else stands between the two, and every read has to be
left in the assembly."""

import os
import re
import subprocess

import pytest

from trellis_quantized_moe_amd.csrc import build as B


def test_gradient_kernel_reads_back_what_other_lanes_may_have_written(tmp_path):
    if not os.path.exists(B.HIPCC):
        pytest.skip("no hipcc")
    with open(os.path.join(B.HERE, "router.hip")) as f:
        src = f.read()
    runtime = "const bool two = p.topk > 16;"
    assert src.count(runtime) == 1
    src = src.replace(runtime, "constexpr bool two = false;")
    host = src.index("// f(blocks of 64")  # one instance instead of the launches
    src = src[:host] + ("template __global__ void route_backward_kernel<1, 3, false>(RouterParams);\n"
                        "}\n}\n")
    hip, asm = tmp_path / "one.hip", tmp_path / "one.s"
    hip.write_text(src)
    r = subprocess.run([B.HIPCC] + B.FLAGS + ["-I" + B.HERE, "-x", "hip", "--cuda-device-only",
                                              "-S", str(hip), "-o", str(asm)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    body = re.search(r"^_ZN4exl3\S*route_backward_kernel\S*:.*?^\.Lfunc_end", asm.read_text(),
                     re.S | re.M).group(0)
    # single values: the chosen logit, the tag, the entry an addition starts from
    assert len(re.findall(r"\bds_read2?_b32\b", body)) >= 3
