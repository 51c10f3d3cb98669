"""What the entry points of gemm_relu_groups.h launch, checked against what the kernels assume.

groups_launches.cpp holds the library's own host code with a recorder in the place of the HIP runtime, so
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
AUTO, TILED, DMA_256, DMA_128, DMA_64, STREAM = -1, 0, 1, 2, 3, 4
COUNTERS = 65536

# Well separated addresses, never followed.
A, B, E, C, D, U, V, W = (i << 44 for i in range(1, 9))


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    so = tmp_path_factory.mktemp("groups_launches") / "groups_launches.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-x", "c++", "-w", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-fno-gnu-unique", "-shared", "-fPIC", "-Wl,-Bsymbolic", os.path.join(HERE, "groups_launches.cpp"),
                    "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.gemm_relu_grouped.argtypes = [vp] * 4 + [i64] * 4 + [ci] * 4 + [vp, i64, vp]
    lib.gemm_relu_grouped_workspace.argtypes = [i64] * 4 + [ci] * 2
    lib.gemm_relu_grouped_backward.argtypes = [vp] * 7 + [i64] * 4 + [ci] * 4 + [vp, i64, vp]
    lib.gemm_relu_grouped_backward_workspace.argtypes = [i64] * 4 + [ci] * 3
    lib.gemm_relu_adapters.argtypes = [vp] * 8 + [i64] * 6 + [ci] * 4 + [vp, i64, vp]
    lib.gemm_relu_adapters_workspace.argtypes = [i64] * 6 + [ci] * 2
    for name in ("grouped", "grouped_backward", "adapters"):
        getattr(lib, f"gemm_relu_{name}_workspace").restype = i64
    lib.launches.restype = ctypes.c_char_p
    return lib


def grouped(host, M, N, K, groups, layout=KN, relu=1, config=AUTO, off=0):
    need = host.gemm_relu_grouped_workspace(M, N, K, groups, 0, layout)
    rc = host.gemm_relu_grouped(A + off, B + off, E, C + off, M, N, K, groups, 0, layout, relu, config, W, need, None)
    return rc, need, json.loads(host.launches())


def backward(host, M, N, K, groups, layout=KN, relu=1, config=AUTO, off=0, need_a=True, need_b=True):
    need = host.gemm_relu_grouped_backward_workspace(M, N, K, groups, 0, layout, relu)
    rc = host.gemm_relu_grouped_backward(D + off, C + off, A + off, B + off, E, U if need_a else None,
                                         V if need_b else None, M, N, K, groups, 0, layout, relu, config, W, need, None)
    return rc, need, json.loads(host.launches())


def check_streams(launches):
    """The streaming and outer kernels take rows as long as the product says: never a copy's pitch."""
    for l in launches:
        if l["kernel"] == "weight_outer":
            assert l["ldp"] == l["i"] and l["ldq"] == l["j"], l
        if l["kernel"] == "rows_skinny":
            layout = l["place"] // 6 % 2
            assert l["lda"] == l["k"] and l["ldb"] == (l["k"] if layout == NK else l["n"]), l


def adapters(host, M, N, K, rank, count, segments, layout=KN, config=AUTO, off=0):
    need = host.gemm_relu_adapters_workspace(M, N, K, rank, count, segments, 0, layout)
    rc = host.gemm_relu_adapters(A + off, B + off, U + off, V + off, D, E, E + (1 << 40), C + off, M, N, K, rank, count,
                                 segments, 0, layout, 1, config, W, need, None)
    return rc, need, json.loads(host.launches())


BLOCKS = (1, 2, 4)                                 # 16-row blocks of the streaming kernels, by their place


def check_places(launches, need):
    """Launches are within the device's limits, and what they write in the workspace is inside it."""
    def inside(at, nbytes, aligned=256):
        assert W + COUNTERS <= at and at + nbytes <= W + need and at % aligned == 0, (l, need)
    for l in launches:
        assert 0 < l["x"] and l["x"] * l["threads"] < 1 << 32 and 0 < l["y"] < 65536 and l["lds"] <= 160 << 10, l
        if l["kernel"] == "mask":
            inside(l["d"], 2 * l["count"])
        elif l["kernel"] == "pad":
            assert l["pitch"] >= l["cols"] and l["pitch"] % 64 == 0
            inside(l["dst"], 2 * l["rows"] * l["pitch"])
        elif l["kernel"] == "rows_skinny" and l["y"] > 1:
            inside(l["parts"], l["x"] * l["y"] * BLOCKS[l["place"] // 12] * 512 * 4)
            assert l["counters"] == W and 4 * l["x"] <= COUNTERS
        elif l["kernel"] == "shrink":
            blocks, chunks = 1 + l["place"] % 2, -(-l["rank"] // 32)
            assert l["rank_pad"] >= l["rank"] and l["rank_pad"] % 64 == 0
            parts = l["x"] * l["y"] * chunks * blocks * 512 * 4 if l["y"] > 1 else 0
            spans = [(l["t"], l["m"] * 2 * l["rank_pad"] * 2), (l["factor"], 4 * l["m"]), (l["row_id"], 4 * l["m"]),
                     (l["part"], parts)]
            for at, nbytes in spans:
                inside(at, nbytes)
            assert all(a + n <= b for (a, n), (b, _) in zip(spans, spans[1:]))
            assert l["counters"] == W and (l["y"] == 1 or 4 * l["x"] <= COUNTERS) and l["lds"] >= chunks * blocks * 512 * 4
            below = l["part"]                       # what lives on until the product has read it
        if l.get("v"):                              # the product after adapter_shrink: its scratch leaves the intermediates
            assert l["kernel"] != "rows_skinny" or l["y"] == 1 or l["parts"] >= below
        if l["kernel"] == "pad" and len(launches) > 1 and launches[0]["kernel"] == "shrink":
            assert l["dst"] >= below


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


# (M, N, K, groups, layout): 17 to 64 rows a group, an odd row length, a long inner dimension.
ODD_STREAMS = [(63, 13089, 1388, 1, NK), (222, 15209, 298, 5, NK), (64, 16385, 960, 1, NK), (32, 50257, 768, 1, NK),
               (64, 12001, 1304, 1, NK), (17, 24001, 2500, 1, NK), (60, 14461, 1316, 1, NK)]


@pytest.mark.parametrize("relu", [0, 1])
@pytest.mark.parametrize("M,N,K,groups,layout", ODD_STREAMS)
def test_backward_never_streams_copies_of_odd_rows(host, M, N, K, groups, layout, relu):
    rc, _, launches = backward(host, M, N, K, groups, layout, relu)
    assert rc == 0 and launches
    check_streams(launches)


def test_streams_take_whole_rows_over_many_sizes(host):
    rng = random.Random(5)
    streamed = padded = 0
    for _ in range(6000):
        if rng.random() < 0.5:
            M, groups = _log(rng, 1, 5000), _log(rng, 1, 128)
            N, K = _log(rng, 1, 60000), _log(rng, 1, 60000)
        else:                                      # around ODD_STREAMS
            groups = rng.randint(1, 6)
            M, N, K = groups * rng.randint(17, 64), _log(rng, 8000, 60000), _log(rng, 200, 2500)
        layout, relu, off = rng.choice([KN, NK]), rng.choice([0, 1]), rng.choice([0, 0, 0, 2])
        config = rng.choice([AUTO] * 5 + [STREAM, DMA_64])
        for call in (grouped, backward):
            rc, _, launches = call(host, M, N, K, groups, layout, relu, config, off)
            assert rc == 0
            check_streams(launches)
            kinds = {l["kernel"] for l in launches}
            streamed += "rows_skinny" in kinds
            padded += "pad" in kinds
    assert streamed > 500 and padded > 500


@pytest.mark.parametrize("tile", [32, 64, 128])
def test_lanes_past_the_last_column_read_inside_v(host, tile):
    # The last rank row of the last adapter ends V: a piece of 4 columns must not pass column N.
    for N in range(4, 400, 4):
        for n in range(0, -(-N // tile) * tile, 4):
            first = host.low_rank_first(n, N, 1)
            assert 0 <= first and first + 4 <= N and (n >= N or first == n), (N, n, first)
    for N in range(1, 200):
        for n in range(0, -(-N // tile) * tile, 4):
            first = host.low_rank_first(n, N, 0)
            assert 0 <= first < N and (n >= N or first == n), (N, n, first)


def test_stream_on_request_is_dAs_alone(host):
    # As the header says: dB goes as by AUTO (one 8192-row group is no work for a lane's loop over rows).
    rng = random.Random(6)
    def plain(launches):
        return [{f: v for f, v in l.items() if f != "c"} for l in launches]
    for _ in range(1500):
        groups = _log(rng, 1, 64)
        args = (_log(rng, 1, 20000), _log(rng, 1, 6000), _log(rng, 1, 6000), groups, rng.choice([KN, NK]), rng.choice([0, 1]))
        off = rng.choice([0, 2])
        rc, _, alone = backward(host, *args, AUTO, off, need_a=False)
        rc_s, _, only_b = backward(host, *args, STREAM, off, need_a=False)
        rc_a, _, only_a = backward(host, *args, STREAM, off, need_b=False)
        rc_2, _, both = backward(host, *args, STREAM, off)
        assert rc == rc_s == rc_a == rc_2 == 0
        assert [l["kernel"] for l in only_a] == ["rows_skinny"] and both[0] == only_a[0], args
        assert only_b == alone and plain(both[1:]) == plain(alone), args
    assert [l["kernel"] for l in backward(host, 8192, 1024, 1024, 1, config=STREAM, relu=0)[2]] == ["rows_skinny", "weight_dma"]


def any_size(rng, top):
    return max(1, min(top, int(round(top ** rng.random())) + rng.choice([-1, 0, 0, 1])))


def test_launches_and_scratch_stay_within_bounds_over_all_sizes(host):
    # Up to the header's limits and the card's memory.
    memory = 288 << 30
    rng = random.Random(7)
    seen = {}
    for i in range(40000):
        top = 1 << 20 if i % 2 else 20000
        M, N, K, groups = any_size(rng, top), any_size(rng, top), any_size(rng, top), any_size(rng, 65535 if i % 2 else 256)
        layout, relu, off = rng.choice([KN, NK]), rng.choice([0, 1]), rng.choice([0, 0, 0, 2])
        config = rng.choice([AUTO] * 6 + [TILED, DMA_256, DMA_128, DMA_64, STREAM])
        rank, count = rng.randint(1, 256), any_size(rng, 65535)
        if 2 * (M * K + groups * K * N + M * N) > memory or 2 * count * rank * (K + N) > memory:
            continue
        for rc, need, launches in (grouped(host, M, N, K, groups, layout, relu, config, off),
                                   backward(host, M, N, K, groups, layout, relu, config, off),
                                   adapters(host, M, N, K, rank, count, groups, layout, config, off)):
            assert rc in (0, -7), rc
            assert rc == 0 or not launches, "refused after a launch"
            check_places(launches, need)
            for l in launches:
                seen[l["kernel"]] = seen.get(l["kernel"], 0) + 1
    assert min(seen.get(k, 0) for k in ("rows_dma", "weight_dma", "rows_skinny", "weight_outer", "mask", "pad", "shrink",
                                        "staged_rows", "staged_grad")) > 100, seen


def test_workspace_sizes_are_what_the_launches_use(host):
    # The copies, the masked gradient, the partial sums and the intermediates, each where it sets the size.
    def up(n):
        return -(-n // 256) * 256
    rc, need, l = grouped(host, 2003, 1101, 2051, 3, NK)
    assert [x["kernel"] for x in l] == ["pad", "pad", "rows_dma"]
    assert need == COUNTERS + up(2 * 2003 * 2112) + up(2 * 3 * 1101 * 2112)     # rows of 2051 to 33 x 64
    rc, need, l = grouped(host, 1, 4096, 4096, 1, KN)
    assert [x["kernel"] for x in l] == ["rows_skinny"] and l[0]["y"] > 1
    assert need == COUNTERS + l[0]["x"] * l[0]["y"] * 512 * 4
    rc, need, l = backward(host, 2003, 1101, 2051, 3, NK)
    assert [x["kernel"] for x in l] == ["pad", "pad", "pad", "rows_dma", "weight_dma"]
    assert need == COUNTERS + up(2 * 2003 * 1152) + up(2 * 2003 * 2112) + up(2 * 3 * 1101 * 2112)
    rc, need, l = backward(host, 8192, 4096, 2048, 16, KN)
    assert [x["kernel"] for x in l] == ["mask", "rows_dma", "weight_dma"] and need == COUNTERS + 2 * 8192 * 4096
    # Rank 12 is kept as 64 entries of two parts; a factor and an adapter for each row; 5 column blocks of
    # rank 130 make 5 blocks of sums a part.
    rc, need, l = adapters(host, 64, 64, 32, 12, 4, 4)
    assert need == COUNTERS + 64 * 64 * 2 * 2 + 64 * 4 + 64 * 4
    rc, need, l = adapters(host, 64, 16384, 8192, 130, 32, 64)
    assert l[0]["kernel"] == "shrink" and l[0]["y"] > 1
    assert need == COUNTERS + 64 * 192 * 2 * 2 + 2 * 64 * 4 + l[0]["x"] * l[0]["y"] * 5 * 512 * 4
