"""The register trade of the 4-bit chunk kernels (no GPU): their warpgroups share out what the block is launched with, so every one of
them has to be compiled to exactly that many registers a thread."""
import os
import re
import subprocess


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "layer_range_stage_gb300", "csrc", "kernels_kv4_chunk.cu")


def test_every_chunk_kernel_has_the_registers_that_it_shares_out(tmp_path):
    from layer_range_stage_gb300 import build as lbuild
    r = subprocess.run([lbuild.nvcc(), *lbuild.ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"),
                        "-Xptxas", "-v", "-c", SRC, "-o", str(tmp_path / "chunk.o")], capture_output=True, text=True, check=True)
    text = open(SRC).read()
    start, soft, prod, rest = (int(re.search(rf"\b{name} = (\d+)", text).group(1)) for name in ("kRegsStart", "kRegsSoft", "kRegsProd", "kRegsRest"))
    assert 8 * soft + 8 * prod + 4 * rest <= 20 * start
    found = re.findall(r"Compiling entry function '(\w+)'.*?Used (\d+) registers", r.stderr, re.S)
    kernels = {name: int(n) for name, n in found if "kv4_chunk_kernel" in name or "kv4_pair_kernel" in name}
    assert len(kernels) == 18 and set(kernels.values()) == {start}, kernels
