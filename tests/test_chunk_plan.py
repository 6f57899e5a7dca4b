"""The chunks of the router's weight gradient, on the CPU: the arithmetic that the kernel
and the workspace take from csrc/chunk_plan.h, compiled by the host's compiler, against
integers without a limit, up to the largest batch that a shape may have."""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mxfp4_routed_expert_gemv_amd", "csrc")
MOST = 2 ** 31 - 1   # pairs of a batch


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host compiler")
    at = tmp_path_factory.mktemp("chunk_plan")
    src, out = at / "plan.cpp", at / "plan.so"
    src.write_text('#include "chunk_plan.h"\n'
                   'extern "C" int chunk() { return k3::kChunk; }\n'
                   'extern "C" int chunks(int n) { return k3::chunks_of(n); }\n'
                   'extern "C" int begin(int q0, int i) { return k3::chunk_begin(q0, i); }\n'
                   'extern "C" int end(int q0, int n, int i) { return k3::chunk_end(q0, n, i); }\n'
                   'extern "C" int most_chunks(int E, long long P) { return k3::most_chunks(E, P); }\n'
                   'extern "C" int most_parts(long long T, long long P) { return k3::most_parts(T, P); }\n')
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(out)], check=True)
    lib = ctypes.CDLL(str(out))
    lib.most_chunks.argtypes = [ctypes.c_int, ctypes.c_longlong]
    lib.most_parts.argtypes = [ctypes.c_longlong, ctypes.c_longlong]
    return lib


def test_chunks_of_an_expert(plan):
    c = plan.chunk()
    for n in (0, 1, c - 1, c, c + 1, 2 * c, 2 * c + 1, 10 ** 6, 2 ** 30, MOST - c, MOST - c + 1, MOST - c + 2, MOST):
        assert plan.chunks(n) == max(-(-n // c), 1), n


@pytest.mark.parametrize("q0,n", [(0, 1), (0, 256), (5, 257), (0, MOST), (1, MOST - 1), (MOST - 1, 1), (MOST, 0),
                                  (MOST - 600, 600), (7, MOST - 7)])
def test_the_last_chunk_ends_with_the_pairs(plan, q0, n):
    c, last = plan.chunk(), plan.chunks(n) - 1
    for i in {0, last // 2, max(last - 1, 0), last}:
        assert plan.begin(q0, i) == q0 + i * c
        assert plan.end(q0, n, i) == min(q0 + (i + 1) * c, q0 + n)
    assert plan.end(q0, n, last) == q0 + n


@pytest.mark.parametrize("counts", [[MOST], [0] * 1023 + [MOST], [MOST // 2 + 1, MOST // 2], [257] * 4, [256] * 4,
                                    [1] * 300, [MOST - 300] + [1] * 300, [257, 0, 1]])
def test_the_workspace_has_room_for_every_chunk(plan, counts):
    # (one slot: every pair is a token of its own)
    T = P = sum(counts)
    chunks = [plan.chunks(n) for n in counts]
    assert sum(chunks) <= plan.most_chunks(len(counts), P)
    assert sum(c for c in chunks if c > 1) <= plan.most_parts(T, P)
