"""Host-side checks at the edges of the operators around the linear: refusals
before any launch (fake pointers, never dereferenced) and which form a call
takes, by its workspace."""
import os
import shutil
import subprocess
import sys

import pytest

A = 0x10000
NULL, SHAPE, ALIGN, ARG = 1, 2, 3, 5


@pytest.fixture(scope="module")
def w8():
    import w8a8_int8_quantized_token_amd as pkg
    return pkg


def test_positions_without_a_rotation_need_a_table_size(w8):
    """rot = 0: P counts where positions are given (rows outside [0, P) are
    padding), and nowhere else."""
    v = (512, 64)

    def call(pos, P, M=0, rot=0):
        return w8.lib.w8a8_qk_norm_rope(A, *v, A, *v, A, A, None, None, pos, A, *v, A, *v, M, P, 4, 2, 64, rot, 1e-6,
                                        0, None)

    def back(pos, P):
        return w8.lib.w8a8_qk_norm_rope_backward(A, *v, A, *v, A, *v, A, *v, A, A, None, None, pos, A, *v, A, *v, None,
                                                 None, 0, P, 4, 2, 64, 0, 1e-6, 0, None, 0, None)

    for P in (0, -1, 2 ** 31):
        assert call(A, P) == back(A, P) == SHAPE and call(None, P) == back(None, P) == 0
        assert call(None, P, rot=16) == SHAPE
    assert call(A, 1) == back(A, 1) == 0
    assert call(A + 2, 4, M=4) == ALIGN


@pytest.mark.parametrize("name", ["linear", "gated_linear"])
def test_which_few_tokens_take_the_few_token_kernel(w8, name):
    """Up to 16 tokens with codes that fit it need no workspace there; many
    channels of a short K are left to the tiled kernel, whose codes do."""
    ws = getattr(w8.lib, f"w8a8_{name}_dynamic_workspace")
    for M in (1, 5, 16):
        for K in (16, 64, 256, 512, 752):
            assert ws(M, 8192 + 16 * K, K) == 0
            assert ws(M, 8192 + 16 * K + 1, K) >= M * K + 4 * M
        assert ws(M, 2 ** 20, 768) == 0


def test_which_linears_are_cut_into_k_ranges(w8):
    """Ranges need slices beside the codes: for K from 6144 on or up to 64
    tokens, where the linear has few tiles."""
    def slices(M, N, K):
        return w8.lib.w8a8_linear_dynamic_workspace(M, N, K) - (M * K + 4 * M + 255) // 256 * 256 >= 8 * M * N

    assert slices(64, 2048, 4096) and slices(33, 512, 5120) and slices(512, 2048, 6144) and slices(256, 2048, 8192)
    assert not slices(65, 2048, 4096) and not slices(512, 2048, 4096) and not slices(256, 512, 6128)


@pytest.mark.parametrize("stale", [False, True])
def test_native_calls_that_are_missing_or_do_not_load(tmp_path, stale):
    name = "w8a8_int8_quantized_token_amd"
    here = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), name)
    shutil.copytree(here, tmp_path / name, ignore=shutil.ignore_patterns("_build", "csrc", "__pycache__", "_calls.so"))
    if stale:
        (tmp_path / name / "_calls.so").write_bytes(b"no library")
    r = subprocess.run([sys.executable, "-c", f"import {name}"], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 1
    assert "ImportError" in r.stderr and "_calls.so is not built or does not load" in r.stderr and "build.py" in r.stderr
