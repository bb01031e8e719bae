"""Host side of the adapter entry points, without a GPU: sizes of the workspace, and calls at the edges
of what they take."""
import subprocess
import sys

import pytest

import bit_weight_only_w2_b200 as lb
from tests.test_adapter_abi import A, adapters, backward, forward


@pytest.mark.parametrize("N,K", [(0, 64), (64, 0), (0, 0)])
def test_workspace_size_of_an_empty_linear(N, K):
    """A linear without rows or columns has a size like any other (a division by its empty K slices ended
    the process, so each is asked for in one of its own)."""
    code = (f"import ctypes; f = ctypes.CDLL({lb.LIB_PATH!r}).lowbit_adapter_workspace_size; f.restype = ctypes.c_size_t; "
            f"f.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] * 2; print(*[f(m, {N}, {K}, l, r) for m in (0, 1, 17, 5000) "
            f"for l, r in ((0, 0), (1, 8), (300, 128))])")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    assert all(int(n) % 256 == 0 for n in r.stdout.split())


@pytest.mark.parametrize("N,K", [(4096, 4096), (9728, 2560), (384, 7680), (136, 256), (9216, 9216)])
@pytest.mark.parametrize("R", [8, 32, 128])
@pytest.mark.parametrize("L", [0, 1, 3, 64, 256, 300, 4096])
def test_workspace_of_a_larger_batch_serves_a_smaller_one(N, K, R, L):
    """The size never falls as the batch grows, through every choice of tile and of K slices."""
    size = lb.load().lowbit_adapter_workspace_size
    sizes = [size(M, N, K, L, R if L else 0) for M in [*range(0, 2400), *range(2400, 41000, 61)]]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_a_linear_without_rows_leaves_nothing_unwritten():
    """N = 0: nothing to do for Y, but P and the 8-bit copy are not empty, so a call that asks for them is
    refused instead of returning OK with both as they were. B is empty then, and may be null."""
    lib = lb.load()
    assert forward(lib, adapters(), N=0, P=A) == 3
    assert forward(lib, adapters(), N=0, codes=A, exps=A) == 3
    assert forward(lib, adapters(B=None), N=0) == 0
    assert forward(lib, adapters(), N=0, M=0, P=A, codes=A, exps=A) == 0
    assert forward(lib, adapters(B=None)) == 1
    assert backward(lib, adapters(B=None), N=0, dB=None) == 3
