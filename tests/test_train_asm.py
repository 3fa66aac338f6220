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


def unpublished_lds_writes(asm):
    """Barriers that an LDS write of the same wave may still be behind: between the two there is neither a wait for
    the LDS counter to reach zero nor another barrier."""
    found, kernel, pending = [], None, None
    for text in (l.split(";")[0].strip() for l in asm.splitlines()):
        if text.startswith("_Z") and text.endswith(":"):
            kernel, pending = text[:-1], None
        elif text.startswith("ds_write"):
            pending = text
        elif text.startswith("s_waitcnt") and "lgkmcnt(0)" in text:
            pending = None
        elif text.startswith("s_barrier"):
            if pending:
                found.append((kernel, pending))
            pending = None
    return found


def test_lds_writes_are_done_before_the_barrier_that_publishes_them(tmp_path):
    """The hardware's barrier does not wait for a wave's own LDS operations."""
    for src in ("fp8gg_bf16.hip", "fp8gg_blocks.hip", "fp8gg_grad.hip", "fp8gg_kernels.hip"):
        asm = device_asm(tmp_path, os.path.join(B.CSRC, src))
        assert "s_barrier" in asm
        found = unpublished_lds_writes(asm)
        assert not found, f"{src}: {len(found)}, first {found[0]}"


def test_the_scan_sees_a_missing_wait():
    bad = "_Zk:\n\tds_write_b64 v1, v[2:3]\n\ts_barrier\n"
    assert unpublished_lds_writes(bad) == [("_Zk", "ds_write_b64 v1, v[2:3]")]
    assert unpublished_lds_writes(bad.replace("\ts_barrier", "\ts_waitcnt lgkmcnt(0)\n\ts_barrier")) == []
    assert unpublished_lds_writes(bad.replace("\ts_barrier", "\ts_waitcnt vmcnt(0)\n\ts_barrier")) != []
