"""Odd widths of the fused residual norm around the forms that its rows take,
and what the backward kernels' registers come to."""

import os
import re
import subprocess

import pytest
import torch

from test_isa_store_hazard import CSRC, HIPCC, ROOT

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [4095, 4096, 4097, 4098, 5001, 6143, 8190, 8191, 8193, 16383])
def test_odd_widths(cols):
    from test_block_norm import check, make
    check(make(2, 11, cols, F32, BF16, F32, seed=cols), "layer", "rms", 0.5)
    check(make(3, 9, cols, BF16, F32, BF16, seed=cols), "rms", "layer", 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [4104, 4097, 8192])
def test_whole_widths_in_unaligned_rows(cols):
    from test_block_norm import check, make
    t = make(1, 9, cols, F32, BF16, F32, seed=cols)
    for n in ("resid", "h"):
        wide = torch.full((1, 9, cols + 40), float("nan"), dtype=t[n].dtype, device="cuda")
        wide[..., 3:3 + cols] = t[n]
        t[n] = wide[..., 3:3 + cols]
    check(t, "rms", "layer", 1.0)


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
def test_backward_rows_up_to_8192_columns_stay_in_registers(tmp_path):
    """A row's columns and their sums in scratch memory cost more than the
    whole pass: 4096 rows of 5001 took as long as elementary torch operations."""
    out = tmp_path / "norm.s"
    cmd = [HIPCC, "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-O3", "-std=c++17",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, "--cuda-device-only", "-S", os.path.join(CSRC, "kernels_norm.hip"),
           "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    found = {}
    for block in out.read_text().split("  - .agpr_count:")[1:]:
        name = re.search(r"norm_bwd_kernelI\w\wLi(\d+)ELi(\d+)ELb", block)
        if name:
            vec, chunks = int(name.group(1)), int(name.group(2))
            spilled = int(re.search(r"\.vgpr_spill_count:\s*(\d+)", block).group(1))
            found[vec, chunks] = max(found.get((vec, chunks), 0), spilled)
    # the widest rows of each form: 64 threads x 4, 1024 x 4, 1024 x 8 and 1024 x 8 in one chunk
    for form in ((1, 4), (1, 8), (8, 1)):
        assert found[form] <= 16, (form, found)


@pytest.mark.gpu
@pytest.mark.parametrize("samples,rows,cols", [(300, 1, 520), (2000, 3, 264), (40, 130, 1000), (129, 8, 64), (127, 9, 64),
                                               (3, 128, 257), (70, 100, 2048)])
def test_many_samples_of_few_rows(samples, rows, cols):
    """Modulation that changes every few rows: the column sums of a sample by
    one wave and by a workgroup, on both sides of what chooses between them."""
    from test_block_norm import check, make
    check(make(samples, rows, cols, F32, BF16, F32, seed=samples), "rms", "layer", 0.5)
