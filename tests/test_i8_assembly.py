"""What the compiler made of the per-token int8 kernels, read from the gfx950
assembly of their source.  Their DMA is written out in assembly, which the
compiler does not see as memory instructions, so two things it would otherwise
see to are checked here: a scalar register that a vector instruction wrote is
read by a memory instruction at least five wait states later, and no kernel
spills vector registers (a reload would wait for every DMA under way)."""
import os
import re
import subprocess

import pytest

from block_quantized_int8_q8_amd import build

pytestmark = pytest.mark.skipif(not os.path.exists(build.hipcc()), reason="needs hipcc")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    out = tmp_path_factory.mktemp("asm") / "i8.s"
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([build.hipcc(), *flags, "--cuda-device-only", "-S", os.path.join(build.CSRC, "i8_kernels.hip"), "-o",
                    str(out)], check=True, capture_output=True)
    text = out.read_text()
    parts = re.split(r"^(_ZN3mmq\S+):\s.*$", text, flags=re.M)
    bodies = {n: b[:b.find(".Lfunc_end")] for n, b in zip(parts[1::2], parts[2::2]) if ".Lfunc_end" in b}
    return bodies, text


def registers(text):
    found = {int(r) for r in re.findall(r"(?<![\w\[:])s(\d+)\b", text)}
    for a, b in re.findall(r"s\[(\d+):(\d+)\]", text):
        found |= set(range(int(a), int(b) + 1))
    return found


def test_scalar_registers_settle_before_dma_reads_them(kernels):
    dma = 0
    for name, body in kernels[0].items():
        written, at = {}, 0                   # scalar register -> wait states passed when a vector instruction wrote it
        for line in body.splitlines():
            line = line.split(";")[0].strip()
            if not line or line.startswith(".") or line.endswith(":"):
                continue
            op = line.split()[0]
            if op.startswith("buffer_"):
                dma += "lds" in line
                for r in registers(line):
                    assert at - written.get(r, -99) >= 5, (name, line)
            at += int(line.split()[1]) + 1 if op == "s_nop" else 1
            dest = re.match(r"\S+\s+(s\[\d+:\d+\]|s\d+)\b", line)
            if dest and op.startswith("v_"):
                written.update((r, at) for r in registers(dest[1]))
            elif dest and op.startswith("s_"):
                for r in registers(dest[1]):
                    written.pop(r, None)
    assert dma > 500                          # the kernels' DMA was seen


def test_no_kernel_spills_vector_registers(kernels):
    spills = re.findall(r"\.name:\s+(_ZN3mmq\S+).*?\.vgpr_spill_count:\s+(\d+)", kernels[1], re.S)
    assert len(spills) >= 60
    assert all(n == "0" for _, n in spills), [k for k, n in spills if n != "0"]
    assert all("scratch_" not in body for body in kernels[0].values())
