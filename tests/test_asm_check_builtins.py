"""The wait states after a builtin MFMA that the build asks for, and the ways through branches that it follows."""
import os

import pytest

from offload_memory_centric_amd import asm_check, build

MFMA = "\tv_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[4:7], v[0:3]"
READ = "\tv_add_f32 v12, v13, v2"
END = "\ts_endpgm"


def findings(*lines):
    return asm_check.gfx950_early_reads(list(enumerate(lines, 1)))


def test_eight_wait_states():
    """As many as the compiler puts between the instruction and a read of its result."""
    for op in ("f16", "bf16"):
        mfma = MFMA.replace("bf16", op)
        assert findings(mfma, "\ts_nop 6", READ) and not findings(mfma, "\ts_nop 7", READ)
    # a form that is not listed has the longest latency's
    slow = "\tv_mfma_f32_32x32x16_f16 v[0:15], v[16:19], v[20:23], v[0:15]"
    assert findings(slow, "\ts_nop 7", "\ts_nop 7", READ) and not findings(slow, "\ts_nop 7", "\ts_nop 7", "\ts_nop 1", READ)


def test_two_jumps_to_a_read():
    """Out of a loop, and on from the block behind it: two jumps between the instruction and the read."""
    out = [".LBB0_1:", MFMA, "\ts_cbranch_scc1 .LBB0_3", "\ts_branch .LBB0_1", ".LBB0_3:", "\ts_branch .LBB0_5", ".LBB0_4:",
           "\tv_mov_b32 v20, v21", ".LBB0_5:"]
    assert findings(*out, READ, END)
    assert findings(*out, "\ts_nop 4", READ, END)
    assert not findings(*out, "\ts_nop 5", READ, END)
    # three, and conditional ones
    ways = [MFMA, "\ts_cbranch_vccz .LBB0_1", END, ".LBB0_1:", "\ts_cbranch_execz .LBB0_2", END, ".LBB0_2:",
            "\ts_cbranch_scc0 .LBB0_3", END, ".LBB0_3:"]
    assert findings(*ways, READ, END)
    assert not findings(*ways, "\ts_nop 4", READ, END)


def test_a_loop_without_a_read_ends():
    assert not findings(".LBB0_1:", "\ts_branch .LBB0_1", MFMA, ".LBB0_2:", "\ts_branch .LBB0_2")
    assert not findings(MFMA, ".LBB0_2:", "\ts_cbranch_scc1 .LBB0_2", END)


def test_a_result_that_is_overwritten_is_followed_from_there():
    again = MFMA.replace("v[0:3], v[8:11]", "v[0:3], v[16:19]")
    assert findings(MFMA, "\ts_nop 7", again, READ)
    assert not findings(MFMA, again, "\ts_nop 7", READ)


def test_built_sources_keep_them():
    for src in build.BUILTIN_SOURCES:
        path = build.device_asm(src)
        if not os.path.exists(path):
            pytest.skip("no kept assembly")
        found = asm_check.check_file(path, check=asm_check.gfx950_early_reads)
        assert found and not any(found.values()), {k: v[:3] for k, v in found.items() if v}


def kernels(tmp_path, check, *texts):
    path = tmp_path / "listing.s"
    path.write_text("".join("_ZN2zi%dk%dEv:\n%s\n.Lfunc_end%d:\n\t.section .rodata\n" % (2, i, t, i) for i, t in enumerate(texts)))
    return asm_check.check_file(str(path), check=check)


@pytest.mark.parametrize("check", [asm_check.check_kernel, asm_check.gfx950_early_reads])
def test_code_behind_the_first_end_is_checked(tmp_path, check):
    """A kernel with an early end has blocks behind it; an end holds nothing up for the block that follows it."""
    early = "\ts_cbranch_scc1 .LBB0_2\n\ts_endpgm\n.LBB0_2:\n"
    good = early + MFMA + "\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n" + READ + "\n\ts_endpgm"
    bad = early + MFMA + "\n" + READ + "\n\ts_endpgm"
    res = kernels(tmp_path, check, good, bad, good)
    assert [bool(v) for v in res.values()] == [False, True, False] and len(res) == 3
    assert not any(kernels(tmp_path, check, MFMA + "\n\ts_endpgm\n.LBB0_3:\n" + READ + "\n\ts_endpgm").values())


def test_two_jumps_in_a_kernel_of_inline_assembly():
    """Its results are read through two branches as late as behind one."""
    out = [MFMA.replace("v[0:3]", "a[0:3]"), "\ts_cbranch_scc1 .LBB0_3", END, ".LBB0_3:", "\ts_branch .LBB0_5", ".LBB0_4:", "\ts_nop 7",
           "\ts_nop 7", "\ts_nop 7", ".LBB0_5:"]
    drain, read = ["\ts_nop 7", "\ts_nop 7"], "\tv_accvgpr_read_b32 v8, a1"
    assert asm_check.check_kernel(list(enumerate(out + [read, END], 1)))
    assert not asm_check.check_kernel(list(enumerate(out + drain + [read, END], 1)))
