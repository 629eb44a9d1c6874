"""Refusals of the group-scaled and routing calls, and the definitions the GPU
tests compare against; no GPU is used and no call here reaches a launch."""
import os
import re

import numpy as np
import pytest
import torch

import binary_weight_transformer_b200 as bwt
import gs_reference as ref

FAKE = 0x10000  # 64 KB-aligned, never dereferenced
INVALID, ALIGN, UNSUPPORTED = bwt.ERR_INVALID_ARG, bwt.ERR_ALIGNMENT, bwt.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from binary_weight_transformer_b200 import _build
    _build.build()
    return bwt.lib()


ARTIFACT = dict(packed=FAKE, ldp=128, s_g=FAKE, sdt=bwt.F32, lds=2, group=128)
BAD_ARTIFACT = [
    (dict(packed=None), INVALID), (dict(s_g=None), INVALID), (dict(sdt=bwt.I32), INVALID), (dict(sdt=7), INVALID),
    (dict(group=0), INVALID), (dict(group=48), INVALID), (dict(group=512), INVALID), (dict(group=-32), INVALID),
    (dict(ldp=112), INVALID), (dict(lds=1), INVALID), (dict(ldp=136), ALIGN), (dict(packed=FAKE + 8), ALIGN),
    (dict(s_g=FAKE + 2), ALIGN), (dict(s_g=FAKE + 1, sdt=bwt.BF16), ALIGN), (dict(K=0), INVALID), (dict(N=0), INVALID),
    (dict(K=-5), INVALID), (dict(N=2**31), INVALID), (dict(K=bwt.GS_MAX_K + 1, ldp=2**20), UNSUPPORTED), (dict(N=2**30 + 1), UNSUPPORTED),
]


@pytest.mark.parametrize("change,want", BAD_ARTIFACT + [
    (dict(w=None), INVALID), (dict(wdt=bwt.I32), INVALID), (dict(ldw=255), INVALID), (dict(w=FAKE + 2), ALIGN),
    (dict(w=FAKE + 1, wdt=bwt.BF16), ALIGN)])
def test_pack_and_unpack_refuse(lib, change, want):
    a = dict(ARTIFACT, w=FAKE, wdt=bwt.F32, N=8, K=256, ldw=256, **{k: v for k, v in change.items() if k not in ARTIFACT and k not in ("w", "wdt", "N", "K", "ldw")})
    a.update(change)
    assert lib.lowbit_gs_pack(a["w"], a["wdt"], a["N"], a["K"], a["ldw"], a["group"], a["packed"], a["ldp"], a["s_g"],
                              a["sdt"], a["lds"], None, None) == want
    assert lib.lowbit_gs_unpack(a["packed"], a["ldp"], a["s_g"], a["sdt"], a["lds"], a["N"], a["K"], a["group"], a["w"],
                                a["wdt"], a["ldw"], None, None) == want


def test_pack_refuses_rows_of_a_gigabyte(lib):
    """The packer writes all of a row's ldp bytes and addresses them in 31 bits."""
    assert lib.lowbit_gs_pack(FAKE, bwt.F32, 8, 256, 256, 128, FAKE, 2 ** 30, FAKE, bwt.F32, 2, None, None) == UNSUPPORTED


TOKENS = dict(q=FAKE, ldq=256, s_x=FAKE, M=4, N=8, K=256, y=FAKE, ydt=bwt.F32, ldy=8)
BAD_TOKENS = [
    (dict(q=None), INVALID), (dict(s_x=None), INVALID), (dict(y=None), INVALID), (dict(M=0), INVALID),
    (dict(M=-1), INVALID), (dict(M=2**31), INVALID), (dict(ldq=240), INVALID), (dict(ldq=264), ALIGN),
    (dict(q=FAKE + 8), ALIGN), (dict(s_x=FAKE + 1), ALIGN), (dict(y=FAKE + 2), ALIGN),
    (dict(y=FAKE + 1, ydt=bwt.BF16), ALIGN), (dict(ydt=bwt.I32), INVALID), (dict(ldy=7), INVALID),
]


@pytest.mark.parametrize("change,want", BAD_ARTIFACT + BAD_TOKENS + [
    (dict(flags=2), INVALID), (dict(flags=8), INVALID)])
def test_linear_refuses(lib, change, want):
    a = {**ARTIFACT, **TOKENS, "flags": 0, **change}
    assert lib.lowbit_gs_linear(a["q"], a["ldq"], a["s_x"], a["M"], a["K"], a["packed"], a["ldp"], a["s_g"], a["sdt"],
                                a["lds"], a["group"], a["N"], a["y"], a["ydt"], a["ldy"], a["flags"], None,
                                None) == want


@pytest.mark.parametrize("change,want", BAD_ARTIFACT + BAD_TOKENS + [
    (dict(offsets=None), INVALID), (dict(E=0), INVALID), (dict(E=bwt.MOE_MAX_EXPERTS + 1), INVALID),
    (dict(ps=8 * 128 - 16), INVALID), (dict(ss=15), INVALID), (dict(ps=8 * 128 + 8), ALIGN),
    (dict(offsets=FAKE + 2), ALIGN)])
def test_experts_refuse(lib, change, want):
    a = {**ARTIFACT, **TOKENS, "offsets": FAKE, "E": 3, "ps": 8 * 128, "ss": 16, **change}
    assert lib.lowbit_gs_linear_experts(a["q"], a["ldq"], a["s_x"], a["M"], a["K"], a["offsets"], a["E"], a["packed"],
                                        a["ldp"], a["ps"], a["s_g"], a["sdt"], a["lds"], a["ss"], a["group"], a["N"],
                                        a["y"], a["ydt"], a["ldy"], None, None) == want


@pytest.mark.parametrize("change,want", [
    (dict(experts=None), INVALID), (dict(offsets=None), INVALID), (dict(pos=None), INVALID), (dict(T=0), INVALID),
    (dict(k=0), INVALID), (dict(T=2**30, k=2), INVALID), (dict(E=0), INVALID), (dict(E=1025), INVALID),
    (dict(experts=FAKE + 4, wide=1), ALIGN), (dict(experts=FAKE + 2), ALIGN), (dict(pos=FAKE + 1), ALIGN),
    (dict(offsets=FAKE + 2), ALIGN)])
def test_plan_refuses(lib, change, want):
    a = {**dict(experts=FAKE, wide=0, T=4, k=2, E=8, offsets=FAKE, pos=FAKE), **change}
    assert lib.lowbit_moe_plan(a["experts"], a["wide"], a["T"], a["k"], a["E"], a["offsets"], a["pos"], None,
                               None) == want


SLOTS = dict(pos=FAKE, T=4, k=2, rows=8)
BAD_SLOTS = [(dict(pos=None), INVALID), (dict(T=0), INVALID), (dict(k=0), INVALID), (dict(rows=0), INVALID),
             (dict(T=2**30, k=2), INVALID), (dict(rows=2**31), INVALID), (dict(pos=FAKE + 2), ALIGN)]


@pytest.mark.parametrize("change,want", BAD_SLOTS + [
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(nb=0), INVALID), (dict(ldx=63), INVALID),
    (dict(ldo=63), INVALID), (dict(s_x=FAKE), INVALID), (dict(s_out=FAKE), INVALID),
    (dict(s_x=FAKE + 2, s_out=FAKE), ALIGN), (dict(s_x=FAKE, s_out=FAKE + 1), ALIGN)])
def test_gather_refuses(lib, change, want):
    a = {**SLOTS, **dict(x=FAKE, nb=64, ldx=64, s_x=None, out=FAKE, ldo=64, s_out=None), **change}
    assert lib.lowbit_moe_gather(a["x"], a["nb"], a["ldx"], a["s_x"], a["pos"], a["T"], a["k"], a["out"], a["ldo"],
                                 a["s_out"], a["rows"], None, None) == want


@pytest.mark.parametrize("change,want", BAD_SLOTS + [
    (dict(ys=None), INVALID), (dict(y=None), INVALID), (dict(dt=bwt.I32), INVALID), (dict(K=0), INVALID),
    (dict(ldys=31), INVALID), (dict(ldy=31), INVALID), (dict(ys=FAKE + 2), ALIGN), (dict(y=FAKE + 1), ALIGN),
    (dict(w=FAKE + 2), ALIGN)])
def test_combine_refuses(lib, change, want):
    a = {**SLOTS, **dict(ys=FAKE, dt=bwt.F32, ldys=32, w=FAKE, K=32, y=FAKE, ldy=32), **change}
    assert lib.lowbit_moe_combine(a["ys"], a["dt"], a["ldys"], a["rows"], a["pos"], a["w"], a["T"], a["k"], a["K"],
                                  a["y"], a["ldy"], None, None) == want


@pytest.mark.parametrize("change,want", BAD_SLOTS + [
    (dict(dy=None), INVALID), (dict(ys=None), INVALID), (dict(w=None), INVALID), (dict(d_ys=None), INVALID),
    (dict(d_w=None), INVALID), (dict(dt=9), INVALID), (dict(K=0), INVALID), (dict(lddy=31), INVALID),
    (dict(ldys=31), INVALID), (dict(ldd=31), INVALID), (dict(dy=FAKE + 2), ALIGN), (dict(ys=FAKE + 2), ALIGN),
    (dict(d_ys=FAKE + 2), ALIGN), (dict(w=FAKE + 2), ALIGN), (dict(d_w=FAKE + 2), ALIGN)])
def test_combine_backward_refuses(lib, change, want):
    a = {**SLOTS, **dict(dy=FAKE, lddy=32, ys=FAKE, ldys=32, dt=bwt.F32, w=FAKE, K=32, d_ys=FAKE, ldd=32, d_w=FAKE),
         **change}
    assert lib.lowbit_moe_combine_backward(a["dy"], a["lddy"], a["ys"], a["ldys"], a["dt"], a["rows"], a["pos"], a["w"],
                                           a["T"], a["k"], a["K"], a["d_ys"], a["ldd"], a["d_w"], None, None) == want


def test_groups(lib):
    assert lib.lowbit_gs_groups(1001, 32) == 32 == bwt.gs_groups(1001, 32)
    assert lib.lowbit_gs_groups(256, 256) == 1
    assert lib.lowbit_gs_groups(0, 32) == 0 and lib.lowbit_gs_groups(64, 33) == 0
    with pytest.raises(ValueError):
        bwt.gs_groups(64, 33)


def test_python_refuses_before_any_call():
    """CPU tensors, wrong types, shapes and strides raise in the wrapper."""
    f, i8, u8, i32 = torch.float32, torch.int8, torch.uint8, torch.int32
    z = lambda *s, d=f: torch.zeros(*s, dtype=d)  # noqa: E731
    for call in (lambda: bwt.lowbit_gs_pack(z(4, 64)),
                 lambda: bwt.lowbit_gs_unpack(z(4, 32, d=u8), z(4, 2), 64, 32),
                 lambda: bwt.lowbit_gs_linear(z(2, 64, d=i8), z(2), z(4, 32, d=u8), z(4, 2), 32),
                 lambda: bwt.lowbit_gs_linear_experts(z(2, 64, d=i8), z(2), z(2, d=i32), z(1, 4, 32, d=u8), z(1, 4, 2), 32),
                 lambda: bwt.lowbit_moe_plan(z(4, 2, d=i32), 8), lambda: bwt.lowbit_moe_gather(z(4, 8), z(4, 2, d=i32)),
                 lambda: bwt.lowbit_moe_combine(z(8, 8), z(4, 2, d=i32)),
                 lambda: bwt.lowbit_moe_combine_backward(z(4, 8), z(8, 8), z(4, 2, d=i32), z(4, 2))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: bwt.lowbit_gs_pack(z(64)), lambda: bwt.lowbit_moe_plan(z(4, d=i32), 8),
                 lambda: bwt.lowbit_moe_gather(z(4), z(4, 2, d=i32))):
        with pytest.raises(ValueError, match="dimension"):
            call()
    for call, name in ((lambda: bwt.lowbit_gs_linear(z(2, 64), z(2), z(4, 32, d=u8), z(4, 2), 32), "int8"),
                       (lambda: bwt.lowbit_gs_pack(z(4, 64, d=torch.float16)), "float16"),
                       (lambda: bwt.lowbit_moe_plan(z(4, 2), 8), "int32 or int64"),
                       (lambda: bwt.lowbit_moe_combine(z(4, 2, d=torch.float64), z(2, 2, d=i32)), "float64")):
        with pytest.raises(TypeError, match=name):
            call()
    with pytest.raises(ValueError, match="F32 or BF16"):
        bwt.lowbit_gs_pack(z(4, 64), 32, bwt.I32)


def test_reference_packing_round_trip():
    codes = np.random.default_rng(0).integers(-7, 8, (3, 37)).astype(np.int8)
    p = ref.pack(codes, 32)
    k = np.arange(37)
    n = (p[:, 4 * (k // 8) + k % 4] >> (4 * (k % 8 // 4))) & 15
    assert np.array_equal(np.where(n > 7, n.astype(int) - 16, n), codes)


def test_reference_quantiser_on_worked_rows():
    """Scale 1: the codes are the weights rounded, halves to even; a group of
    zeros has scale 0; the second group has its own scale."""
    w = np.zeros((1, 64), np.float32)
    w[0, :7] = [7, 0.5, 1.5, -2.5, 6.5, -0.49, 3]
    w[0, 32:35] = [-14, 1, 3]
    codes, s = ref.quantise(w, 32, False)
    assert s.tolist() == [[1.0, 2.0]]
    assert codes[0, :7].tolist() == [7, 0, 2, -2, 6, 0, 3]
    assert codes[0, 32:35].tolist() == [-7, 0, 2]


def test_reference_plan_on_a_worked_table():
    off, pos = ref.plan(np.array([[2, 0], [-1, 2], [0, 2]]), 3)
    assert off.tolist() == [0, 2, 2, 5]
    assert pos.tolist() == [[2, 0], [-1, 3], [1, 4]]


def test_registers():
    """The tcgen05 kernel splits its registers after launch (256 threads of 64,
    256 of 192), which needs the 128 per thread that it is compiled for; the
    packer runs at 2048 threads per SM."""
    from binary_weight_transformer_b200 import _build
    _build.build()
    seen = {"gs_gemm": 0, "gs_pack": 0}
    for name, regs, spill in (("gs_gemm", 128, 16), ("gs_pack", 32, 8)):
        path = os.path.join(os.path.dirname(_build.__file__), "_build", name + ".cu.ptxas.txt")
        if not os.path.exists(path):
            pytest.skip("no ptxas report (library built elsewhere)")
        for m in re.finditer(r"Compiling entry function '([^']+)'.*?(\d+) bytes spill stores.*?Used (\d+) registers",
                             open(path).read(), re.S):
            if name + "_kernel" in m.group(1):
                seen[name] += 1
                assert int(m.group(2)) <= spill, m.group(1)
                assert int(m.group(3)) == regs if name == "gs_gemm" else int(m.group(3)) <= regs, m.group(1)
    assert seen == {"gs_gemm": 16, "gs_pack": 32}
