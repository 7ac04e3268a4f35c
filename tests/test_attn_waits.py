"""Bounded waits of the attention kernels, as their source has them (no GPU
needed): each lane of a warp has its own clock, so a wait that decides whether a
warp goes on has to be agreed on before instructions that want the whole warp."""
import os
import re

from pre_rope_kv_gb300 import build as kbuild


def source(name):
    with open(os.path.join(kbuild.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_decoding_step_agrees_on_its_waits():
    loop = source("kvi_attn_decode4.cu").split("for (int it = 0; it < pairs; ++it)")[1].split("__any_sync")[0]
    waits = re.findall(r"[^\n]*\bmbar_wait\w*\([^\n]*", loop)
    assert len(waits) == 1 and "__all_sync(0xffffffffu, mbar_wait(" in waits[0]


def test_warps_come_together_before_aligned_instructions():
    """Lanes that went their own way (a lane's own store, a column's own rescaling) meet before a barrier or
    matrix instruction that wants the warp as one."""
    tile = source("kvi_attn_tile.cu")
    before = tile.split('asm volatile("bar.sync 3, 128;"')[0].rstrip().removesuffix("if (i == 0)").rstrip()
    assert before.endswith("__syncwarp();")
    announce = tile.split("void announce(uint64_t &bar)")[1].split("template")[0]
    assert "@q mbarrier.arrive" in announce and "if (" not in announce
    softmax = tile.split("setmaxnreg.inc")[1]
    wait = softmax.split("tl.s_full[i]")[1].split("break;")[0].rstrip()
    assert wait.endswith("__syncwarp();")
    assert re.search(r"sum \*= f;\s*}\s*__syncwarp\(\);\s*if \(j > 0\)", softmax)
    assert re.search(r"\+= inf - inf;\s*}\s*__syncwarp\(\);\s*}", softmax)
    for name in ("kvi_attn_prompt.cu", "kvi_attn_decode4.cu"):
        rescale = source(name).split("if (__any_sync(0xffffffffu, move)) {")[1].split("pack_bf16(p0, p1)")[0]
        assert re.search(r"\*= f;\s*}\s*}\s*__syncwarp\(\);\s*}", rescale), name
    added = source("kvi_attn_prompt.cu").split("if (__any_sync(0xffffffffu, bad != 0)) {")[1].split("mma16816")[0]
    assert re.search(r"\+= x;\s*}\s*__syncwarp\(\);\s*}", added)


def test_nothing_is_read_as_read_only():
    """These kernels begin while the previous one may still write what they read."""
    for name in ("kvi_attn.cuh", "kvi_attn_prompt.cu", "kvi_attn_tile.cu", "kvi_attn_decode4.cu", "kvi_attn_join.cu", "kvi_cache4.cu"):
        assert not re.search(r"__ldg\b|ld\.global\.nc", source(name)), name
