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
