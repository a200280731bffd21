"""The operators between the linears are set up one by one: what one of them
lacks on a device is not refused by the others."""

import os
import shutil
import subprocess

import pytest
import torch

import gpu_helpers as H

pytestmark = pytest.mark.gpu


def test_norms_and_rope_do_not_need_the_attention_kernels_registers(tmp_path, monkeypatch):
    """A build whose attention kernels are short of the registers that their
    warps share out, as another compiler's might be: attention is refused
    before anything is launched, norms and rotary positions run."""
    from nvfp4_w4a4_quantized_smooth_b200 import build
    build.build()
    s = H.svdq()
    src = tmp_path / "csrc"
    shutil.copytree(build.CSRC, src)
    path = src / "ka_attention.cuh"
    text = path.read_text()
    assert "SOFTMAX_REGS = 208" in text
    path.write_text(text.replace("SOFTMAX_REGS = 208", "SOFTMAX_REGS = 216"))
    lib = str(tmp_path / "libsvdq_few_registers.so")
    r = subprocess.run([build.find_nvcc(), *build.NVCC_FLAGS, "-Xptxas", "-O1", "-I", build.INCLUDE, "-I", str(src),
                        os.path.join(str(src), "svdq.cu"), "-o", lib], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]

    x, y = (torch.randn(5, 256, device="cuda").bfloat16() for _ in range(2))
    q = x.view(5, 2, 128)
    pos = torch.zeros(5, 3, dtype=torch.int32, device="cuda")
    plan = s.RopePlan((32, 48, 48), 256.0, 128)
    want = s.norm_gate_residual(x, y), s.rope_qk(q, None, pos, plan)[0]
    monkeypatch.setattr(s, "_lib", s.load_library(lib))
    for _ in range(2):
        with pytest.raises(s.SvdqError) as e:
            s.attention(q, q, q)
        assert e.value.status == s.SVDQ_ERR_UNSUPPORTED
        got = s.norm_gate_residual(x, y), s.rope_qk(q, None, pos, plan)[0]
        s.check_device_error()
    for a, b in ((got[0][0], want[0][0]), (got[0][1], want[0][1]), (got[1], want[1])):
        assert (a.float() - b.float()).abs().max() <= 2.0 ** -7 * b.float().abs().max()
