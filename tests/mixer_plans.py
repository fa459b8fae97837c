"""How csrc/mixer_plans.hpp splits sizes over workgroups, read from a small host build of it."""
from __future__ import annotations

import ctypes
import functools
import os
import subprocess
import tempfile

from tests.conftest import ROOT

SOURCE = r"""
#include "mixer_plans.hpp"
extern "C" {
int recurrence_group(int64_t B, int64_t L, int64_t D, int es) { return ssm::recurrence::group_of(B, L, D, es); }
void conv_plan(int64_t B, int64_t L, int64_t D, int width, int es, int64_t *out) {
  const ssm::conv::BwdPlan p = ssm::conv::bwd_plan(B, L, D, width, es);
  out[0] = p.nrow, out[1] = p.nchunk, out[2] = p.nruns, out[3] = p.ctiles;
}
void heads_plan(int64_t B, int64_t L, int heads, int d, int rot, int bwd, int es, int64_t *out) {
  const ssm::heads::Plan p = ssm::heads::plan_of(B, L, heads, d, rot, bwd != 0, es);
  out[0] = p.rows, out[1] = p.tsub, out[2] = p.nchunk, out[3] = p.nruns, out[4] = p.nblk, out[5] = p.hb;
}
}
"""


@functools.lru_cache(maxsize=None)
def _lib():
    folder = tempfile.mkdtemp()
    so, src = os.path.join(folder, "plans.so"), os.path.join(folder, "plans.cpp")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC",
                    "-I", os.path.join(ROOT, "selective_state_space_10_amd", "csrc"), src, "-o", so], check=True)
    lib = ctypes.CDLL(so)
    I, J = ctypes.c_int64, ctypes.c_int
    lib.recurrence_group.argtypes = [I, I, I, J]
    lib.conv_plan.argtypes = [I, I, I, J, J, ctypes.POINTER(I)]
    lib.heads_plan.argtypes = [I, I, J, J, J, J, J, ctypes.POINTER(I)]
    return lib


def recurrence_group(B, L, D, es):
    """Chunks of 128 steps per published state."""
    return _lib().recurrence_group(B, L, D, es)


def conv_backward(B, L, D, width, es):
    """Steps that a wave walks over for a chunk, chunks of a row, workgroups of a tile of channels, such tiles."""
    out = (ctypes.c_int64 * 4)()
    _lib().conv_plan(B, L, D, width, es, out)
    return dict(zip(("nrow", "nchunk", "nruns", "ctiles"), out))


def heads(B, L, heads, d, rot, bwd, es):
    """Rows of a group between two fillings of the angles, tokens at once, chunks of tokens, workgroups of a block of
    heads, such blocks, heads of one."""
    out = (ctypes.c_int64 * 6)()
    _lib().heads_plan(B, L, heads, d, rot, bwd, es, out)
    return dict(zip(("rows", "tsub", "nchunk", "nruns", "nblk", "hb"), out))
