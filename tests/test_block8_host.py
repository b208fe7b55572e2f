"""CPU checks of the 8-bit products' C ABI (include/moe_block8.h): what is
refused before anything touches a device, the padded row count, and the
direct-load rule of the compiled kernels (M0 is set in the same statement as
each load and used by nothing else)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
NULL = ctypes.c_void_p(0)
FAKE = ctypes.c_void_p(1 << 20)
OFF8 = ctypes.c_void_p((1 << 20) + 8)
OFF1 = ctypes.c_void_p((1 << 20) + 1)


@pytest.fixture(scope="module")
def moe():
    import combine_dispatch_amd as m
    if not os.path.exists(m.LIB_PATH):
        from combine_dispatch_amd import build
        build.build()
    m.lib()
    return m


def test_padded_rows(moe):
    assert moe.moe_padded_rows(0, 1) == 0
    assert moe.moe_padded_rows(1, 1) == 128
    assert moe.moe_padded_rows(128, 1) == 128
    assert moe.moe_padded_rows(129, 1) == 256
    # every division of R rows into E groups fits
    for R, sizes in ((10, [1] * 10), (300, [129, 1, 170]), (5, [0, 5, 0])):
        need = sum((n + 127) // 128 * 128 for n in sizes)
        assert need <= moe.moe_padded_rows(R, len(sizes)) < need + 128 * len(sizes)
    assert moe.moe_padded_rows(-1, 1) == 0 and moe.moe_padded_rows(1, 0) == 0 and moe.moe_padded_rows(1, 1025) == 0


def test_quantise_rows_arguments(moe):
    f = moe.lib().moe_quantise_rows
    assert f(0, 64, 0, NULL, NULL, NULL, NULL, NULL) == moe.MOE_OK
    assert f(-1, 64, 0, FAKE, NULL, FAKE, FAKE, NULL) == moe.MOE_ERR_INVALID_ARG
    assert f(4, 0, 0, FAKE, NULL, FAKE, FAKE, NULL) == moe.MOE_ERR_INVALID_ARG
    assert f(4, 64, 5, FAKE, NULL, FAKE, FAKE, NULL) == moe.MOE_ERR_INVALID_ARG
    assert f(4, (1 << 20) + 1, 0, FAKE, NULL, FAKE, FAKE, NULL) == moe.MOE_ERR_UNSUPPORTED
    assert f((1 << 28) + 1, 64, 0, FAKE, NULL, FAKE, FAKE, NULL) == moe.MOE_ERR_UNSUPPORTED
    for bad in ((NULL, FAKE, FAKE), (FAKE, NULL, FAKE), (FAKE, FAKE, NULL), (OFF1, FAKE, FAKE), (FAKE, OFF8, FAKE)):
        assert f(4, 64, 1, bad[0], NULL, bad[1], bad[2], NULL) == moe.MOE_ERR_INVALID_ARG


def test_quantise_weights_arguments(moe):
    f = moe.lib().moe_quantise_weights
    assert f(0, 8, 8, 0, FAKE, FAKE, FAKE, NULL, NULL, NULL) == moe.MOE_ERR_INVALID_ARG
    assert f(65536, 8, 8, 0, FAKE, FAKE, FAKE, NULL, NULL, NULL) == moe.MOE_ERR_UNSUPPORTED
    assert f(1, 8, 8, 0, FAKE, FAKE, FAKE, FAKE, NULL, NULL) == moe.MOE_ERR_INVALID_ARG  # codes_t alone
    assert f(1, 8, 8, 0, FAKE, FAKE, FAKE, NULL, FAKE, NULL) == moe.MOE_ERR_INVALID_ARG
    assert f(1, 8, 8, 0, FAKE, OFF8, FAKE, NULL, NULL, NULL) == moe.MOE_ERR_INVALID_ARG


def test_quantise_columns_arguments(moe):
    f = moe.lib().moe_quantise_columns
    assert f(0, 8, 1, 0, NULL, NULL, NULL, NULL, NULL) == moe.MOE_OK
    assert f(4, 8, 2, 0, FAKE, NULL, FAKE, FAKE, NULL) == moe.MOE_ERR_INVALID_ARG  # groups without offsets
    assert f(4, 8, 1025, 0, FAKE, FAKE, FAKE, FAKE, NULL) == moe.MOE_ERR_UNSUPPORTED
    assert f(4, 8, 1, 0, FAKE, NULL, OFF8, FAKE, NULL) == moe.MOE_ERR_INVALID_ARG


def test_products_arguments(moe):
    L, S = moe.lib(), moe.MoeBlockShape
    g, wg = L.moe_block_gemm, L.moe_block_gemm_wgrad
    assert g(S(0, 8, 128, 1), NULL, NULL, NULL, NULL, NULL, NULL, NULL) == moe.MOE_OK
    assert g(S(4, 8, 100, 1), FAKE, FAKE, FAKE, FAKE, NULL, FAKE, NULL) == moe.MOE_ERR_UNSUPPORTED
    for s in (S(-1, 8, 128, 1), S(4, 0, 128, 1), S(4, 8, 0, 1), S(4, 8, 128, 0), S(4, 8, 128, 2)):
        assert g(s, FAKE, FAKE, FAKE, FAKE, NULL, FAKE, NULL) == moe.MOE_ERR_INVALID_ARG
        assert wg(s, FAKE, FAKE, FAKE, FAKE, NULL, FAKE, NULL) == moe.MOE_ERR_INVALID_ARG
    for s in (S((1 << 28) + 1, 8, 128, 1), S(4, (1 << 20) + 1, 128, 1), S(4, 8, 1 << 21, 1), S(4, 8, 128, 1025)):
        assert g(s, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, NULL) == moe.MOE_ERR_UNSUPPORTED
        assert wg(s, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, NULL) == moe.MOE_ERR_UNSUPPORTED
    assert wg(S((1 << 23) + 1, 8, 8, 1), FAKE, FAKE, FAKE, FAKE, NULL, FAKE, NULL) == moe.MOE_ERR_UNSUPPORTED
    s = S(4, 8, 128, 1)
    ok = [FAKE] * 4
    for i in range(4):
        args = list(ok)
        args[i] = NULL
        assert g(s, *args, NULL, FAKE, NULL) == moe.MOE_ERR_INVALID_ARG
        assert wg(s, *args, NULL, FAKE, NULL) == moe.MOE_ERR_INVALID_ARG
    assert g(s, *ok, NULL, NULL, NULL) == moe.MOE_ERR_INVALID_ARG
    assert wg(s, *ok, NULL, NULL, NULL) == moe.MOE_ERR_INVALID_ARG
    assert g(s, OFF8, FAKE, FAKE, FAKE, NULL, FAKE, NULL) == moe.MOE_ERR_INVALID_ARG
    assert g(s, FAKE, FAKE, OFF8, FAKE, NULL, FAKE, NULL) == moe.MOE_ERR_INVALID_ARG
    assert g(s, *ok, NULL, OFF1, NULL) == moe.MOE_ERR_INVALID_ARG
    assert wg(s, OFF8, FAKE, FAKE, FAKE, NULL, FAKE, NULL) == moe.MOE_ERR_INVALID_ARG


def test_binding_refuses_host_tensors(moe):
    u = lambda *s: torch.zeros(s, dtype=torch.uint8)
    f = torch.zeros
    with pytest.raises(moe.MoeError, match="GPU"):
        moe.moe_quantise_rows(f(4, 8), u(4, 128), f(1, 4))
    with pytest.raises(moe.MoeError, match="GPU"):
        moe.moe_quantise_weights(f(1, 4, 8), u(1, 4, 128), f(1, 1, 1))
    with pytest.raises(moe.MoeError, match="GPU"):
        moe.moe_quantise_columns(f(4, 8), u(8, 128), u(1, 8))
    with pytest.raises(moe.MoeError, match="GPU"):
        moe.moe_block_gemm(u(4, 128), f(1, 4), u(1, 8, 128), f(1, 1, 1), f(4, 8).bfloat16())
    with pytest.raises(moe.MoeError, match="GPU"):
        moe.moe_block_gemm_wgrad(u(8, 128), u(1, 8), u(8, 128), u(1, 8), f(1, 8, 8).bfloat16(), rows=4)


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    out = str(tmp_path_factory.mktemp("asm") / "block_gemm.s")
    cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "--cuda-device-only", "-S", "-Xclang",
           "-target-feature", "-Xclang", "-packed-fp32-ops", "-o", out,
           os.path.join(ROOT, "combine_dispatch_amd", "csrc", "block_gemm.hip")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return open(out).read().splitlines()


def test_m0_is_only_written_by_the_direct_loads(asm):
    implicit = re.compile(r"\b(s_set_gpr_idx_\w+|s_movrel\w*|v_movrel\w*|s_sendmsg\w*|ds_gws\w*|"
                          r"v_interp\w*|ds_\w+_addtid\w*|s_ttracedata)\b")
    insts = [s for s in (l.split(";")[0].strip() for l in asm) if s and not s.startswith(".") and not s.endswith(":")]
    loads = 0
    for i, s in enumerate(insts):
        if re.search(r"\bm0\b", s):
            assert re.match(r"^s_mov_b32 m0, s\d+$", s), s
        assert not implicit.search(s), s
        if s.startswith("global_load_lds_"):
            loads += 1
            assert insts[i - 1] == "s_nop 0" and insts[i - 2].startswith("s_mov_b32 m0,"), insts[i - 3:i + 1]
    assert loads > 20


def test_no_packed_fp32_and_no_spills(asm):
    assert not any(re.match(r"\s*v_pk_(add|mul|fma)_f32", l) for l in asm)
    scratch = [int(l.split()[-1]) for l in asm if l.strip().startswith(".amdhsa_private_segment_fixed_size")]
    assert scratch and not any(scratch)
