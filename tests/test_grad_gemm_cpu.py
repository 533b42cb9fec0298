"""Host checks of the W8A8 linear's gradients, and their workspace sizes, without a GPU."""
import ctypes as C

import pytest
import torch

import int8_w8a8_quantized_smoothed_b200 as w8
from int8_w8a8_quantized_smoothed_b200 import build as w8build

A = 0x10000  # a 16-byte aligned fake address; the host checks never dereference it


@pytest.fixture(scope="module")
def L():
    w8build.build()
    return w8.lib()


def _p(i, off=0):
    return None if i is None else C.c_void_p(A + i * 0x100000 + off)


@pytest.mark.parametrize("name", ["dgrad", "dgrad_fp8", "wgrad", "wgrad_fp8", "dgrad_silu",
                                  "dgrad_silu_fp8"])
def test_host_checks(L, name):
    fn = getattr(L, "w8a8_gemm_" + name)
    silu = "silu" in name

    def call(dy=_p(0), q=_p(1), s=_p(2), M=4, N=64, K=128, gu=_p(3), out=_p(4), ws=_p(5),
             n=1 << 28):
        return fn(dy, q, s, M, N, K, *((gu,) if silu else ()), out, ws, n, None)

    for missing in ("dy", "q", "s", "out") + (("gu",) if silu else ()):
        assert call(**{missing: None}) == -1, missing
    assert call(M=0) == -1 and call(N=0) == -1 and call(K=8) == -1
    assert call(N=12) == -3 and call(K=24) == -3
    assert call(M=(1 << 30) + 1) == -3 and call(N=1 << 31) == -3 and call(K=1 << 31) == -3
    for bad in ("dy", "q", "out", "ws") + (("gu",) if silu else ()):
        assert call(**{bad: _p(6, 8)}) == -2, bad
    assert call(out=_p(0)) == -1 and call(out=_p(1)) == -1
    if silu:
        assert call(out=_p(3)) == -1
    if not torch.cuda.is_available():
        assert call() == -7


def test_workspace_sizes(L):
    d, wg = L.w8a8_gemm_dgrad_workspace_size, L.w8a8_gemm_wgrad_workspace_size
    tile = 2 * 256 * 256 * 4  # two partial tiles per CTA pair
    narrow = 2 * 16 * 128 * 4  # and per CTA of the kernel for up to 16 rows
    assert d(1, 64, 256) == 0                       # one k-block: nothing to split
    assert d(16, 2048, 128) == 8 * narrow           # 32 k-blocks, four for each CTA
    assert d(17, 2048, 128) == 16 * narrow          # of 32 rows
    assert d(4, 12, 64) == 0 and d(0, 64, 64) == 0  # refused shapes
    assert d(1, 4096, 4096) == 148 * narrow         # 32 tiles of 64 k-blocks on 148 SMs
    assert d(129, 4096, 256) == 16 * tile           # 64 k-blocks, four for each pair
    assert d(4096, 72, 4096) == 72 * 4096 * 2       # many rows: the bf16 weight
    assert wg(72, 4096, 4096) == 72 * 4096 * 2      # or the bf16 activations; short sums whole
    assert wg(4096, 256, 256) == 16 * tile
    # the bf16 operand (to 256 bytes), then the partial tiles of a split
    assert d(4100, 8184, 272) == 8184 * 272 * 2 + 68 * tile
    assert d(4100, 8200, 272) == 68 * tile          # longer sums are converted by the kernel
    assert d(265, 7880, 4400) == 72 * 2 * tile      # in tiles of 512 rows


def test_binding_refuses_cpu_tensors():
    dy = torch.zeros(4, 64, dtype=torch.bfloat16)
    q = torch.zeros(64, 128, dtype=torch.int8)
    with pytest.raises(ValueError, match="CUDA"):
        w8.w8a8_gemm_dgrad(dy, q, torch.ones(64))
    with pytest.raises(ValueError, match="CUDA"):
        w8.w8a8_gemm_dgrad(dy=dy, wq=q, s_ch=torch.ones(64))
    with pytest.raises(TypeError, match="dy must be"):
        w8.w8a8_gemm_wgrad(None, q, torch.ones(64))
