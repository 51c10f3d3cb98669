"""What the entry points of gemm_relu_blocks.h launch, checked against what the kernels assume.

blocks_launches.cpp holds the library's own host code with a recorder in the place of the HIP runtime, so
argument checks, kernel choice, workspace places and launch shapes run as they are, without a GPU.
"""
import ctypes
import json
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
KN, NK = 0, 1
COUNTERS = 65536
TOO_LARGE = -7
MEMORY = 288 << 30

# Well separated addresses, never followed.
A, SA, B, SB, E, C, D, U, V, W = (i << 44 for i in range(1, 11))


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    so = tmp_path_factory.mktemp("blocks_launches") / "blocks_launches.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-x", "c++", "-w", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-fno-gnu-unique", "-shared", "-fPIC", "-Wl,-Bsymbolic", os.path.join(HERE, "blocks_launches.cpp"),
                    "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.gemm_relu_quantize_blocks.argtypes = [vp] * 6 + [i64] * 5 + [ci] * 4 + [vp]
    lib.gemm_relu_blocks.argtypes = [vp] * 6 + [i64] * 6 + [ci] * 6 + [vp]
    lib.gemm_relu_blocks_backward.argtypes = [vp] * 8 + [i64] * 5 + [ci] * 5 + [vp, i64, vp]
    lib.gemm_relu_blocks_backward_workspace.argtypes = [i64] * 3
    lib.gemm_relu_experts.argtypes = [vp] * 9 + [i64] * 8 + [ci] * 4 + [vp, i64, vp]
    lib.gemm_relu_experts_workspace.argtypes = [i64] * 5 + [ci]
    lib.gemm_relu_blocks_backward_workspace.restype = lib.gemm_relu_experts_workspace.restype = i64
    lib.launches.restype = ctypes.c_char_p
    return lib


def whole(n, unit):
    return -(-n // unit) * unit


def nb(n):
    return -(-n // 128)


def quantize(host, count, R, C_, rows=True, transposed=True, tiles=0, off=0):
    rc = host.gemm_relu_quantize_blocks(A + off, None, B if rows else None, SA, C if transposed else None, SB, count, R, C_,
                                        whole(C_, 16), whole(R, 16), 1, 0, tiles, 0, None)
    return rc, json.loads(host.launches())


def product(host, M, N, K, groups=0, b_rows=False, config=-1):
    rc = host.gemm_relu_blocks(A, SA, B, SB, E if groups else None, C, M, N, K, max(groups, 1), whole(K, 16), whole(K, 16), 0, 1,
                               0 if b_rows else 1, 1, 1, config, None)
    return rc, json.loads(host.launches())


def backward(host, M, N, K, need_x=True, need_w=True, formats=(0, 0)):
    need = host.gemm_relu_blocks_backward_workspace(M, N, K)
    rc = host.gemm_relu_blocks_backward(D, C, A, SA, B, SB, U if need_x else None, V if need_w else None, M, N, K, whole(M, 16),
                                        whole(N, 16), 1, *formats, 1, 1, W, need, None)
    return rc, need, json.loads(host.launches())


def experts(host, tokens, N, K, hidden, count, top, layout=NK, eight=False, routed=True, off=0):
    need = host.gemm_relu_experts_workspace(tokens, N, hidden, count, top, layout)
    rc = host.gemm_relu_experts(A + off, B, SA if eight else None, C, SB if eight else None, E if routed else None, U, V, D, tokens, N,
                                K, hidden, count, top, whole(K, 16), whole(hidden, 16), 1, 1, 0 if eight else -1, layout, W,
                                max(need, 0), None)
    return rc, need, json.loads(host.launches())


STREAM_ROWS, STREAM_COLS, TILES = (16, 16, 16, 32, 32, 64), (32, 64, 64, 64, 64, 64), (256, 128, 64)


def check(launches):
    for l in launches:
        assert l["kernel"] != "unknown"
        assert 0 < l["x"] and l["x"] * l["threads"] < 1 << 32 and l["y"] == 1 and l["lds"] <= 32 << 10, l


def any_size(rng, top):
    return max(1, min(top, int(round(top ** rng.random())) + rng.choice([-1, 0, 0, 1])))


def test_quantizer(host):
    rng, apart = random.Random(1), 0
    for i in range(20000):
        top = 1 << 20 if i % 2 else 6000
        count, R, C_ = any_size(rng, 65535 if i % 4 == 1 else 3), any_size(rng, top), any_size(rng, top)
        if 4 * count * R * C_ > MEMORY:
            continue
        rows, transposed = rng.choice([(True, True), (True, False), (False, True)])
        rc, launches = quantize(host, count, R, C_, rows, transposed, rng.choice([0, 1]), rng.choice([0, 0, 2]))
        assert rc in (0, TOO_LARGE) and len(launches) == (rc == 0)
        check(launches)
        tiles = count * nb(R) * nb(C_)
        for l in launches:
            assert (l["tiles_r"], l["tiles_c"]) == (nb(R), nb(C_)) and bool(l["q"]) == rows and bool(l["qt"]) == transposed
            # a workgroup for each tile, or one for each direction of it
            assert (l["apart"], l["x"]) in ((0, tiles), (tiles, 2 * tiles)) and (not l["apart"] or (rows and transposed))
            apart += l["apart"] > 0
    assert apart > 100


def test_products(host):
    rng, seen = random.Random(2), {}
    for i in range(40000):
        top = 1 << 20 if i % 2 else 6000
        M, N, K = any_size(rng, top), any_size(rng, top), any_size(rng, top)
        groups = rng.choice([0, any_size(rng, 65535 if i % 2 else 200)])
        config = rng.choice([-1] * 5 + [0, 1, 2, 3])
        if M * K + max(groups, 1) * N * K + 2 * M * N > MEMORY:
            continue
        rc, launches = product(host, M, N, K, groups, rng.choice([True, False]), config)
        assert rc in (0, TOO_LARGE) and len(launches) == (rc == 0)
        check(launches)
        for l in launches:
            heavy = min(max(groups, 1), M) * N * whole(K, 16) >= 96 << 20
            if l["kernel"] == "stream":
                r, c = STREAM_ROWS[l["place"]], STREAM_COLS[l["place"]]
                # every group may end in a partial tile, and rows of no group may follow
                assert l["x"] == (min(M, M // r + groups + 1) if groups else -(-M // r)) * -(-N // c) and l["once"] == heavy
                assert config in (-1, 3)
            else:
                # (a stream of more workgroups than a launch has goes to tiles)
                assert l["kernel"] == "tile" and l["x"] <= 512 and (config in (-1, 3) or l["place"] == config)
                assert l["once"] == (heavy and (groups > 0 or M <= TILES[l["place"]]) and l["place"] != 0)
            seen[l["kernel"], l["place"]] = seen.get((l["kernel"], l["place"]), 0) + 1
    assert len(seen) >= 8 and min(n for place, n in seen.items() if place != ("stream", 5)) > 20, seen
    # few columns of long sums: 64 rows in one workgroup a CU
    assert [(l["kernel"], l["place"]) for l in product(host, 64, 16384, 8192)[1]] == [("stream", 5)]


def test_backward(host):
    rng, pairs = random.Random(3), 0
    for i in range(20000):
        top = 1 << 20 if i % 4 == 1 else 6000
        M, N, K = any_size(rng, top), any_size(rng, top), any_size(rng, top)
        if 4 * (M * N + M * K + N * K) > MEMORY:
            continue
        rc, need, both = backward(host, M, N, K)
        assert rc in (0, TOO_LARGE)
        check(both)
        if rc:
            continue
        q = both[0]
        assert q["kernel"] == "quantize" and need == host.gemm_relu_blocks_backward_workspace(M, N, K)
        spans = [(q["q"], M * q["ldq"]), (q["s"], 4 * M * nb(N)), (q["qt"], N * q["ldqt"]), (q["st"], 4 * N * nb(M))]
        assert spans[0][0] >= W + COUNTERS and all(at % 256 == 0 for at, _ in spans)
        assert all(at + n <= b for (at, n), (b, _) in zip(spans, spans[1:])) and spans[3][0] + spans[3][1] <= W + need
        if both[1]["kernel"] == "pair":
            pairs += 1
            p = both[1]
            assert len(both) == 2 and p["x"] == p["blocks_x"] + p["blocks_w"] and p["blocks_x"] % 8 == 0 and p["x"] <= 4 * 256 + 16
            assert (p["x_m"], p["x_n"], p["x_k"], p["w_m"], p["w_n"], p["w_k"]) == (M, K, N, N, K, M)
            assert (p["x_a"], p["x_sa"], p["w_a"], p["w_sa"]) == tuple(at for at, _ in spans) and (p["x_c"], p["w_c"]) == (U, V)
            tiles = ("tile", 2)
        else:
            assert [(l["a"], l["c"]) for l in both[1:]] == [(q["q"], U), (q["qt"], V)]
            tiles = None
        # one gradient alone, or of operands of two formats: the same kernels
        _, _, x = backward(host, M, N, K, need_w=False)
        _, _, w = backward(host, M, N, K, need_x=False)
        _, _, mixed = backward(host, M, N, K, formats=(0, 1))
        assert len(x) == len(w) == 2 and not x[0]["qt"] and not w[0]["q"]
        kernels = [(l["kernel"], l["place"]) for l in (x[1], w[1])]
        assert kernels == ([tiles, tiles] if tiles else [(l["kernel"], l["place"]) for l in both[1:]])
        assert [(l["kernel"], l["place"]) for l in mixed[1:]] == kernels
    assert pairs > 300


def test_experts(host):
    rng, seen = random.Random(4), set()
    for i in range(40000):
        wide = i % 4 == 0
        tokens, count = any_size(rng, 64), any_size(rng, 1024)
        top = rng.randint(1, min(16, count))
        N, K, hidden = (any_size(rng, 1 << 20 if wide else 9000) for _ in range(3))
        eight = rng.choice([False, True])
        layout = NK if eight else rng.choice([KN, NK])
        if (1 if eight else 2) * count * hidden * (K + N) > MEMORY:
            continue
        routed, off = rng.choice([True, False]), rng.choice([0, 0, 2])
        rc, need, launches = experts(host, tokens, N, K, hidden, count, top, layout, eight, routed, off)
        assert rc in (0, TOO_LARGE) and (rc == 0 or not launches)
        check(launches)
        if rc:
            assert need == TOO_LARGE
            continue
        first, second = [l for l in launches if l["kernel"] == "experts"]
        assert len(launches) == 2 + (launches[0]["kernel"] == "route")
        # the choices are made once: apart, or by the first product
        assert [bool(l["logits"]) for l in launches] == ([routed, False, False] if len(launches) == 3 else [routed, False])
        slots = tokens * top
        mid, part = second["mid"], second["part"]
        assert mid >= W + COUNTERS and mid + 4 * slots * second["mid_row"] <= part and second["mid_row"] >= hidden
        assert part + 4 * slots * second["splits"] * N <= W + need and part % 256 == 0
        store, odd, which, kind = ((second["place"] // n) % m for n, m in ((8, 4), (4, 2), (2, 2), (1, 2)))
        assert which == 1 and first["place"] // 2 % 2 == 0 and store == (2 if eight else 0 if layout == NK else 1)
        columns = 64 if layout == KN or kind == 1 else 32
        assert second["counters"] == W and 4 * -(-N // columns) <= COUNTERS
        assert 1 <= second["splits"] <= 256 and first["splits"] == 1 and first["x"] <= 768 and second["x"] <= 768
        assert (first["in"], first["out"], second["in"], second["out"]) == (K, hidden, hidden, N)
        odd_1 = off != 0 or K % 2 or (layout == KN and not eight and hidden % 2)
        assert first["place"] // 4 % 2 == bool(odd_1)
        assert odd == bool(not eight and (N if layout == KN else hidden) % 2)
        seen |= {first["place"], second["place"]}
    # 8-bit e4m3 here: 3 storages x odd or not x product x kind, but no odd rows of 8-bit weights in the second
    assert len(seen) >= 22, sorted(seen)
