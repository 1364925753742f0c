"""The inline assembly that the scan sums and broadcasts rows of lanes with, as compiled
for gfx950 (no GPU needed): where a caller passes equal values, what is read last does
not share a register with what is written first."""
import importlib.util
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.join(os.path.dirname(HERE), "recurrent_state_update_amd")

SOURCE = """
#include "dl_ssm_bwd.hip"
namespace dl {
__global__ void equal_row_sums(float *out, const float *in)
{
    float p[16];
    for (int i = 0; i < 16; ++i)
        p[i] = in[i % 8 * 64 + threadIdx.x];
    out[threadIdx.x] = row_sums(p, threadIdx.x % 16);
}
__global__ void equal_fma_bcast(float *out, const float *in)
{
    float acc[8], v[8];
    for (int i = 0; i < 8; ++i)
        acc[i] = v[i] = in[i * 64 + threadIdx.x];
    fma_bcast<0>(acc, v[0], v);
    for (int i = 0; i < 8; ++i)
        out[i * 64 + threadIdx.x] = acc[i];
}
__global__ void equal_fma_bcast_sum(float *out, const float *in)
{
    float v[8];
    for (int i = 0; i < 8; ++i)
        v[i] = in[i * 64 + threadIdx.x];
    float even = v[7], odd = v[6];
    fma_bcast_sum<0>(even, odd, v[0], v);
    out[threadIdx.x] = even + odd;
}
} // namespace dl
"""


def build_module():
    spec = importlib.util.spec_from_file_location("_deltalog_build", os.path.join(PKG, "_build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    b = build_module()
    if shutil.which(b.HIPCC) is None:
        pytest.skip("no hipcc")
    src = tmp_path_factory.mktemp("rows") / "equal.hip"
    src.write_text(SOURCE)
    r = subprocess.run([b.HIPCC, *b.CFLAGS, "-S", "--cuda-device-only", str(src), "-o", "-"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return r.stdout


def block(assembly, kernel):
    """(written, read, read) registers of each instruction of the kernel's block."""
    body = re.search(rf"^_ZN2dl\d+{kernel}E.*?:.*?s_endpgm", assembly, re.S | re.M).group()
    asm, = (b for b in re.findall(r"#ASMSTART\n(.*?)#ASMEND", body, re.S) if "_dpp" in b)
    return re.findall(r"v_\w+_dpp (v\d+), (v\d+), (v\d+)", asm)


def test_row_sums(assembly):
    ops = block(assembly, "equal_row_sums")
    assert len(ops) == 24
    first, then = ops[:8], ops[8:16]  # in place; from the other eight
    assert len({d for d, _, _ in first}) == 8 and all(d == a == b for d, a, b in first)
    assert not {d for d, _, _ in first} & {r for _, a, b in then for r in (a, b)}


@pytest.mark.parametrize("kernel,sums", [("equal_fma_bcast", 8), ("equal_fma_bcast_sum", 2)])
def test_sums_of_products(assembly, kernel, sums):
    ops = block(assembly, kernel)
    assert len(ops) == 8
    written = {d for d, _, _ in ops}
    assert len(written) == sums
    assert not written & {r for _, a, b in ops for r in (a, b)}
