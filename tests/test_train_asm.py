"""CPU check of the generated gfx950 code of the bf16 products: like the fp8 kernels, they copy to LDS
with M0 loaded right before each copy, and touch M0 nowhere else."""
import os

from fp8_rowwise_scaled_amd import build as B
from tests.test_kernel_asm import device_asm, m0_uses_outside_lds_copies


def test_products_use_m0_only_for_the_lds_copies(tmp_path):
    asm = device_asm(tmp_path, os.path.join(B.CSRC, "fp8gg_bf16.hip"))
    assert "global_load_lds" in asm and "ds_read_b64_tr_b16" in asm and "v_mfma_f32_16x16x32_bf16" in asm
    uses = m0_uses_outside_lds_copies(asm)
    assert not uses, f"M0 used outside the LDS copies: {uses[:5]}"


def test_no_packed_fp32(tmp_path):
    for src in ("fp8gg_bf16.hip", "fp8gg_blocks.hip", "fp8gg_grad.hip"):
        asm = device_asm(tmp_path, os.path.join(B.CSRC, src))
        assert not any(i in asm for i in ("v_pk_add_f32", "v_pk_mul_f32", "v_pk_fma_f32")), src
