"""Every argument of the two products of gemm_relu_blocks_backward, in one launch or in two, against the formulas:
dX (M, K) = D (M, N) @ WT (K, N)^T and dW (N, K) = D^T (N, M) @ XT (K, M)^T.  On the CPU, with a recorder."""
import ctypes
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
COUNTERS = 65536
DC, C, XT, SXT, WT, SWT, DX, DW, W = (i << 44 for i in range(1, 10))
NAMES = ("formats", "b_rows", "pair", "a", "sa", "b", "sb", "c", "ends", "m", "n", "k", "groups", "lda", "ldb", "relu", "bf16")


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    so = tmp_path_factory.mktemp("blocks_arguments") / "blocks_arguments.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-x", "c++", "-w", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-fno-gnu-unique", "-shared", "-fPIC", "-Wl,-Bsymbolic", os.path.join(HERE, "blocks_arguments.cpp"),
                    "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.gemm_relu_blocks_backward.argtypes = [vp] * 8 + [i64] * 5 + [ci] * 5 + [vp, i64, vp]
    lib.gemm_relu_blocks_backward_workspace.argtypes = [i64] * 3
    lib.gemm_relu_blocks_backward_workspace.restype = i64
    return lib


def whole(n, unit):
    return -(-n // unit) * unit


def products(host):
    out = (ctypes.c_int64 * 170)()
    return [dict(zip(NAMES, out[17 * i:17 * i + 17])) for i in range(host.products(out, 10))]


def expected(M, N, K, ldxt, ldwt, fmt, fx, fw, bf16):
    """The two products, with the workspace as the quantizer leaves it: Q, its scales, Q^T, its scales."""
    ldq, ldqt = (whole(n, 16 if n <= 1024 else 128) for n in (N, M))
    q = W + COUNTERS
    s = q + whole(M * ldq, 256)
    qt = s + whole(4 * M * -(-N // 128), 256)
    st = qt + whole(N * ldqt, 256)
    common = {"ends": 0, "groups": 1, "relu": 0, "bf16": bf16}
    return (dict(common, formats=2 * fmt + fw, b_rows=0, a=q, sa=s, b=WT, sb=SWT, c=DX, m=M, n=K, k=N, lda=ldq, ldb=ldwt),
            dict(common, formats=2 * fmt + fx, b_rows=1, a=qt, sa=st, b=XT, sb=SXT, c=DW, m=N, n=K, k=M, lda=ldqt, ldb=ldxt))


def test_arguments(host):
    rng, seen = random.Random(5), {}
    sizes = [(2048, 512, 512), (2100, 1500, 2100), (4100, 2056, 4100), (1, 16384, 8192), (8192, 4096, 4096), (100, 200, 300)]
    while len(sizes) < 4000:
        sizes.append(tuple(max(1, int(9000 ** rng.random())) for _ in range(3)))
    for i, (M, N, K) in enumerate(sizes):
        fmt, fx, fw, bf16 = (i >> b & 1 for b in range(4))
        ldxt, ldwt = whole(M, 16) + 16 * rng.randint(0, 3), whole(N, 16) + 16 * rng.randint(0, 3)
        need = host.gemm_relu_blocks_backward_workspace(M, N, K)
        both = expected(M, N, K, ldxt, ldwt, fmt, fx, fw, bf16)
        for want_x, want_w in ((True, True), (True, False), (False, True)):
            assert host.gemm_relu_blocks_backward(DC, C, XT, SXT, WT, SWT, DX if want_x else None, DW if want_w else None, M, N, K, ldxt,
                                                  ldwt, fmt, fx, fw, bf16, 1, W, need, None) == 0
            got = products(host)
            pair = [p.pop("pair") for p in got]
            assert got == [p for p, wanted in zip(both, (want_x, want_w)) if wanted], (M, N, K)
            assert len(set(pair)) == 1 and (not pair[0] or (len(got) == 2 and fx == fw))
            seen[pair[0], len(got)] = seen.get((pair[0], len(got)), 0) + 1
    assert min(seen.get(p, 0) for p in ((1, 2), (0, 2), (0, 1))) > 300, seen
