"""Launches of calls that share a workspace, on the CPU: those of one call follow each other, whichever threads and
entry points share the buffer, and calls with other workspaces go on meanwhile.

workspace_launches.cpp is a recorder in the place of the HIP runtime; the entry points are the library's own.
"""
import ctypes
import os
import subprocess
import threading

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "tiled_dense_gemm_relu_amd", "csrc")

# Well separated addresses, never followed.
A, SA, B, SB, E, C, D, U, V, W, W2 = (i << 42 for i in range(1, 12))
ROOM = 1 << 34


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    so = tmp_path_factory.mktemp("workspace_launches") / "workspace_launches.so"
    sources = [os.path.join(HERE, "workspace_launches.cpp")] + [os.path.join(CSRC, s) for s in (
        "gemm_relu_api.hip", "groups_api.hip", "blocks_api.hip")]
    subprocess.run(["g++", "-std=c++17", "-O1", "-x", "c++", "-w", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-pthread",
                    "-I" + os.path.join(os.path.dirname(HERE), "include"), "-D__align__(n)=", "-DHIP_SYMBOL(s)=s", "-fno-gnu-unique", "-shared", "-fPIC",
                    "-Wl,-Bsymbolic", *sources, "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.gemm_relu_splitk.argtypes = [vp] * 3 + [i64] * 3 + [ci] * 4 + [vp, i64, vp]
    lib.gemm_relu_grouped.argtypes = [vp] * 4 + [i64] * 4 + [ci] * 4 + [vp, i64, vp]
    lib.gemm_relu_grouped_backward.argtypes = [vp] * 7 + [i64] * 4 + [ci] * 4 + [vp, i64, vp]
    lib.gemm_relu_adapters.argtypes = [vp] * 8 + [i64] * 6 + [ci] * 4 + [vp, i64, vp]
    lib.gemm_relu_blocks_backward.argtypes = [vp] * 8 + [i64] * 5 + [ci] * 5 + [vp, i64, vp]
    lib.gemm_relu_experts.argtypes = [vp] * 9 + [i64] * 8 + [ci] * 4 + [vp, i64, vp]
    lib.launched.argtypes = [ci, ci, ctypes.c_double]
    return lib


def calls(host, ws):
    """Every entry point that takes a workspace, at sizes that use it: name -> (call, launches)."""
    return {
        "splitk": (lambda: host.gemm_relu_splitk(A, B, C, 64, 256, 8192, 0, 0, -1, 4, ws, ROOM, None), 1),
        "grouped, streamed": (lambda: host.gemm_relu_grouped(A, B, E, C, 8, 512, 8192, 4, 0, 1, 1, -1, ws, ROOM, None), 1),
        "grouped, copies": (lambda: host.gemm_relu_grouped(A, B, E, C, 4000, 4001, 4001, 2, 0, 1, 1, -1, ws, ROOM, None), 3),
        "grouped_backward": (lambda: host.gemm_relu_grouped_backward(D, C, A, B, E, U, V, 4096, 2048, 2048, 4, 0, 0, 1, -1, ws, ROOM, None), 3),
        "adapters": (lambda: host.gemm_relu_adapters(A, B, U, V, SA, E, D, C, 512, 1024, 1024, 16, 4, 4, 0, 0, 1, -1, ws, ROOM, None), 2),
        "blocks_backward": (lambda: host.gemm_relu_blocks_backward(D, C, A, SA, B, SB, U, V, 4096, 2048, 2048, 4096, 2048, 1, 0, 0, 1, 1, ws, ROOM, None), 3),
        "experts": (lambda: host.gemm_relu_experts(A, B, None, C, None, E, U, V, D, 24, 512, 512, 512, 16, 2, 0, 0, 1, 1, -1, 1, ws, ROOM, None), 3),
    }


def taken(host):
    out = (ctypes.c_int * 100000)()
    return list(out[: host.taken(out, len(out))])


def test_each_call_launches_as_listed(host):
    for name, (call, launches) in calls(host, W).items():
        host.begin(5)
        assert call() == 0, name
        assert taken(host) == [5] * launches, name


def test_launches_of_a_call_stay_together(host):
    """Each entry point on a thread of its own, all with one workspace, many times over."""
    table, rounds, failed = calls(host, W), 60, []

    def run(i, call):
        for n in range(rounds):
            host.begin(i * rounds + n)
            if call() != 0:
                failed.append(i)
    threads = [threading.Thread(target=run, args=(i, call)) for i, (call, _) in enumerate(table.values())]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    log, names, wrong = taken(host), list(table), set()
    assert not failed and len(log) == rounds * sum(n for _, n in table.values())
    for at, call in enumerate(log):
        if at and log[at - 1] != call and call in log[max(0, at - 64):at]:
            wrong.add(names[call // rounds])
    assert not wrong, f"other launches within calls of {sorted(wrong)}"


@pytest.mark.parametrize("first", ["grouped_backward", "adapters", "grouped, copies", "blocks_backward", "experts"])
def test_a_call_waits_for_its_workspace_only(host, first):
    """While a call's first launch waits for a full queue, others with its workspace wait, and all with another go on."""
    taken(host)
    host.hold(1)

    def run(i, call):
        host.begin(i)
        call()
    same, other = calls(host, W), calls(host, W2)
    threads = [threading.Thread(target=run, args=(1, same[first][0]))]
    threads[0].start()
    try:
        assert host.launched(1, 1, 10.0)
        for i, (call, launches) in enumerate(other.values()):
            threads.append(threading.Thread(target=run, args=(10 + i, call)))
            threads[-1].start()
            assert host.launched(10 + i, launches, 5.0), "a call with another workspace was held up"
        for i, (call, _) in enumerate(same.values()):
            threads.append(threading.Thread(target=run, args=(30 + i, call)))
            threads[-1].start()
        late = [name for i, name in enumerate(same) if host.launched(30 + i, 1, 0.1)]
        assert not late, f"{late} launched within a call with the same workspace"
    finally:
        host.hold(-1)
        for t in threads:
            t.join()
    log = [c for c in taken(host) if c == 1 or c >= 30]
    assert log[: same[first][1]] == [1] * same[first][1] and len(log) == same[first][1] + sum(n for _, n in same.values())
