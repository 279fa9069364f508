"""The built code of the BF16 and 4-bit products and of gradient clipping: no scratch, no wide store whose data (the second
operand of a global store, the first of a buffer store) is rewritten at once, and in the BF16 products the wait
states around the MFMAs that are inline assembly (the 256 x 256 tiles, whose accumulators are pinned to AGPRs):
those that the scan of `test_mfma_hazard` knows, and two between a VALU write of an accumulator and the MFMA that adds
to it (of equal accumulators the compiler once kept one and copied it to the others just ahead of their first
MFMA, which then added to what the register held before)."""

import os
import re
import subprocess

import pytest

import test_mfma_hazard as mfma

SOURCES = ["gemm_bf16.hip", "grad_clip.hip", "w4.hip"]


def accumulator_copies(asm):
    """MFMAs within two instructions of a VALU write of their accumulator (straight-line code)."""
    bad, recent = [], []
    for raw in asm.split("\n"):
        line = raw.split(";")[0].strip()
        if not line or line.startswith(".") or line.endswith(":"):
            continue
        op, ops = mfma._split(line)
        wait = int(ops[0]) + 1 if op == "s_nop" else 1
        if op.startswith("v_mfma"):
            acc = mfma._regs(ops[0], "a")
            if any(acc & regs for regs, _ in recent):
                bad.append(line)
        recent = [(regs, w + wait) for regs, w in recent if w + wait < 2]
        if op.startswith("v_accvgpr") and ops:
            recent.append((mfma._regs(ops[0], "a"), 0))
    return bad


def rewritten_data(asm):
    """Stores of 12 or 16 bytes a lane whose data the next instruction writes."""
    bad, wide = [], None
    for raw in asm.split("\n"):
        line = raw.split(";")[0].strip()
        if not line or line.startswith(".") or line.endswith(":"):
            continue
        op, ops = mfma._split(line)
        if wide and op.startswith("v_") and ops and wide[1] & mfma._regs(ops[0], "v"):
            bad.append((wide[0], line))
        m = re.match(r"(buffer|global|flat|scratch)_store_dwordx[34]$", op)
        wide = (line, mfma._regs(ops[0 if m.group(1) == "buffer" else 1], "v")) if m else None
    return bad


def test_scan_finds_rewritten_data():
    store = "\tglobal_store_dwordx4 v[50:51], v[46:49], off offset:16\n"
    assert len(rewritten_data(store + "\tv_mov_b32_e32 v47, 0\n")) == 1
    assert rewritten_data(store + "\tv_mov_b32_e32 v50, 0\n") == [] == rewritten_data(store + "\ts_nop 1\n\tv_mov_b32_e32 v47, 0\n")


def test_scan_finds_a_copied_accumulator():
    asm = "\tv_accvgpr_mov_b32 a4, a0\n\tv_mfma_f32_32x32x16_bf16 a[0:15], v[8:11], v[16:19], a[0:15]\n"
    assert len(accumulator_copies(asm)) == 1
    assert accumulator_copies(asm.replace("\tv_mfma", "\ts_nop 1\n\tv_mfma")) == []


@pytest.fixture(scope="module", params=SOURCES)
def compiled(request, tmp_path_factory):
    from moe_grouped_scaled_amd.build import FLAGS, HIPCC
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("asm") / "k.s"
    flags = [f for f in FLAGS if not f.startswith("-W")]
    res = subprocess.run([HIPCC, *flags, "--cuda-device-only", "-S", os.path.join(mfma.CSRC, request.param), "-o", str(out),
                          "-Rpass-analysis=kernel-resource-usage"], check=True, stdout=subprocess.PIPE,
                         stderr=subprocess.STDOUT, text=True)
    return out.read_text(), res.stdout


def test_no_scratch_and_no_store_hazard(compiled):
    asm, usage = compiled
    names = re.findall(r"Function Name: (\S+)", usage)
    scratch = [int(v) for v in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", usage)]
    assert names and len(names) == len(scratch)
    assert not [(n, s) for n, s in zip(names, scratch) if s]
    assert not rewritten_data(asm)[:5]


def test_large_tiles_keep_their_wait_states(compiled):
    asm, _ = compiled
    if "gemm_bf16_kernel" not in asm:
        return  # no inline MFMAs
    kernels = re.findall(r"^(_Z\w+):[^\n]*\n(.*?)^\.Lfunc_end", asm, flags=re.M | re.S)
    large = [(n, b) for n, b in kernels if re.search(r"gemm_bf16_kernelILi\dELi\dELi4EE", n)]
    assert len(large) == 5
    for name, body in large:
        assert not mfma.violations(body)[:5], name
        assert not accumulator_copies(body)[:5], name
