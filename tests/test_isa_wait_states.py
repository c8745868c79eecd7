"""The built library's gfx950 code keeps the distances between a write of a scalar register and the memory
instruction that reads it, in the inline assembly of the direct loads to LDS as well."""
import os
import shutil

import pytest

from linear_rnn_amd import wkv
from tests import isa_lint, isa_waits

pytestmark = pytest.mark.skipif(not shutil.which(os.path.join(isa_lint.LLVM, "llvm-objdump")),
                                reason="ROCm LLVM tools not installed")


def _parse(body):
    lines = [l.strip() for l in body.strip().splitlines()]
    text = "0000000000000000 <f>:\n" + "".join("\t%s // %012X: 00000000\n" % (l, 4 * n) for n, l in enumerate(lines))
    return isa_waits.instructions(text)["f"]


def test_lint_flags_a_descriptor_word_read_too_early():
    near = """
        v_readfirstlane_b32 s26, v68
        s_add_i32 s46, s46, s57
        s_mov_b32 m0, s46
        s_nop 0
        buffer_load_dword v102, s[24:27], 0 offen lds
    """
    assert [f[1:] for f in isa_waits.close_pairs(_parse(near))] == [("buffer_load_dword", "v_readfirstlane_b32", 3)]
    assert isa_waits.close_pairs(_parse(near.replace("s_nop 0", "s_nop 1"))) != []
    assert isa_waits.close_pairs(_parse(near.replace("s_nop 0", "s_nop 2"))) == []
    assert isa_waits.close_pairs(_parse(near.replace("s26", "s28"))) == []  # not the descriptor's


def test_lint_flags_m0_set_right_before_a_load_to_lds():
    near = """
        s_mov_b32 m0, s4
        global_load_lds_dwordx4 v[2:3], off
    """
    assert [f[1:] for f in isa_waits.close_pairs(_parse(near))] == [("global_load_lds_dwordx4", "s_mov_b32", 0)]
    assert isa_waits.close_pairs(_parse(near.replace("s4\n", "s4\n s_nop 0\n"))) == []
    assert isa_waits.close_pairs(_parse(near.replace("global_load_lds_dwordx4 v[2:3], off",
                                                     "buffer_load_dword v1, s[8:11], 0 offen"))) == []


def test_lint_follows_branches():
    # the write at the loop's bottom is one branch away from the load at its top
    loop = """
        buffer_load_dword v1, s[8:11], 0 offen
        v_mov_b32_e32 v2, v3
        v_mov_b32_e32 v2, v3
        v_mov_b32_e32 v2, v3
        v_mov_b32_e32 v2, v3
        v_readfirstlane_b32 s10, v4
        s_cbranch_scc1 65529
    """
    assert [f[1:] for f in isa_waits.close_pairs(_parse(loop))] == [("buffer_load_dword", "v_readfirstlane_b32", 1)]
    assert isa_waits.close_pairs(_parse(loop.replace("65529", "0"))) == []


KERNELS = ("linattn_state_kernel", "linattn_out16_kernel", "linattn_grad_kernel", "wkv7_scan_kernel")


@pytest.fixture(scope="module")
def built(tmp_path_factory):
    assert os.path.exists(wkv.LIB_PATH), "build the library first"
    out = {}
    for t in isa_lint.disassemble(wkv.LIB_PATH, str(tmp_path_factory.mktemp("isa"))):
        out.update(isa_waits.instructions(t))
    return out


@pytest.mark.parametrize("kernel", KERNELS)
def test_built_kernels_with_direct_loads(built, kernel):
    mine = {n: i for n, i in built.items() if kernel in n}
    assert any(isa_waits._to_lds(mn, ops) for i in mine.values() for _, mn, ops in i)  # not vacuous
    assert [(n, f) for n, i in mine.items() for f in isa_waits.close_pairs(i)] == []


def test_every_built_kernel(built):
    assert [(n, f) for n, i in built.items() for f in isa_waits.close_pairs(i)] == []
