"""Launch grids of the embedding, the block-scaled matrices, the dense layer and
the gradient norm at the ends of the sizes that they accept (no GPU): the library
runs against a runtime that only writes launches down, in a process of its own.

A launch holds fewer than 2^32 threads and at least one; a call that passes its
checks launches nothing that the runtime would refuse."""
import ctypes
import json
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

RUNTIME = r"""
#include <stddef.h>
#include <stdint.h>
typedef struct { uint32_t x, y, z; } size3;
static struct { size3 grid, block; size_t lds; void* stream; } next;
static uint64_t count, blocks[1 << 20], threads[1 << 20];
int __hipPushCallConfiguration(size3 grid, size3 block, size_t lds, void* stream) {
    next.grid = grid; next.block = block; next.lds = lds; next.stream = stream;
    return 0;
}
int __hipPopCallConfiguration(size3* grid, size3* block, size_t* lds, void** stream) {
    *grid = next.grid; *block = next.block; *lds = next.lds; *stream = next.stream;
    return 0;
}
int hipLaunchKernel(const void* f, size3 grid, size3 block, void** args, size_t lds, void* stream) {
    if (count < 1 << 20) {
        blocks[count] = (uint64_t)grid.x * grid.y * grid.z;
        threads[count++] = (uint64_t)block.x * block.y * block.z;
    }
    return 0;
}
int hipFuncSetAttribute(const void* f, int attribute, int value) { return 0; }
int hipGetLastError(void) { return 0; }
void clear(void) { count = 0; }
uint64_t launches(void) { return count; }
uint64_t blocks_of(uint64_t i) { return blocks[i]; }
uint64_t threads_of(uint64_t i) { return threads[i]; }
"""

A = 0x10000          # addresses that nothing reads
ROOM = 1 << 60       # a workspace for any size


def run(runtime):
    """In the process of its own: every call's status and launches, as JSON."""
    rt = ctypes.CDLL(runtime, mode=ctypes.RTLD_GLOBAL)  # before the library, whose symbols it answers
    for name in ("launches", "blocks_of", "threads_of"):
        getattr(rt, name).restype = ctypes.c_uint64
    rt.blocks_of.argtypes = rt.threads_of.argtypes = [ctypes.c_uint64]
    sys.path.insert(0, ROOT)
    from sketched_parameter_sharing_amd import _lib
    lib, byref = _lib.load(), ctypes.byref
    types = {"bf16": _lib.BF16, "f32": _lib.F32}

    def T(rows, cols, dtype="bf16"):
        return byref(_lib.Tensor(A, types[dtype], 0, rows, cols))

    def Q(rows, cols, block=1):
        return byref(_lib.Fp8BlocksView(A, A, rows, cols, block, 0))

    out = {}

    def call(name, function, *args):
        rt.clear()
        status = getattr(lib, function)(*args)
        out[name] = [status, [[rt.blocks_of(i), rt.threads_of(i)] for i in range(rt.launches())]]

    for (R, C) in QUANTIZE:
        for dtype in types:
            x = T(R, C, dtype)
            call(f"quantize {R} {C} {dtype} q", "ss1_quantize_fp8_blocks", x, Q(R, C), None, None)
            call(f"quantize {R} {C} {dtype} qt", "ss1_quantize_fp8_blocks", x, None, Q(C, R), None)
            call(f"quantize {R} {C} {dtype} both", "ss1_quantize_fp8_blocks", x, Q(R, C, 128), Q(C, R, 128), None)
    for M, V, K in EMBEDDING:
        tokens = byref(_lib.Tokens(A, M, 4, 0))
        for dtype in types:
            call(f"forward {M} {V} {K} {dtype}", "ss1_embedding_forward", tokens, T(V, K, dtype), 1.0, T(M, K), None)
            for add in (0, 1) if M < 1 << 30 else ():
                call(f"backward {M} {V} {K} {dtype} {add}", "ss1_embedding_backward", T(M, K, dtype), tokens, 1.0, add,
                     T(V, K), A, ROOM, None)
    for M, N, K in PRODUCTS:
        for dtype in types:
            call(f"matmul {M} {N} {K} {dtype}", "ss1_matmul_fp8_blocks", Q(M, K), Q(N, K, 128), T(M, N, dtype), A, ROOM,
                 None)
            call(f"dense {M} {N} {K} {dtype}", "ss1_dense_forward_fp8", T(M, K, dtype), Q(N, K, 128), T(M, N, dtype),
                 Q(K, M), A, ROOM, None)
            if max(M, N) < 1 << 23:  # the gradients' reductions
                call(f"gradients {M} {N} {K} {dtype}", "ss1_dense_backward_fp8", T(M, N, dtype), Q(K, M), Q(K, N, 128),
                     T(M, K, dtype), T(N, K), A, ROOM, None)
    for chunks in (1, 2048, 2049, (1 << 31) - 1):
        for name in ("ss1_gradnorm", "ss1_gradnorm_clip"):
            call(f"{name} {chunks}", name, A, 3, A, chunks, 1.0, A, A, A, ROOM, None)
    print(json.dumps(out))


MANY = (1 << 31) - 1
# [R][C]: up to 2^24 - 1 tiles of 128 x 128, and either side of 2^23 of them
QUANTIZE = [(1, 1), (1, 1 << 30), (1 << 30, 1), (1, (1 << 30) - 128), (1, (1 << 30) + 1), (1, MANY - 128),
            (MANY - 128, 128), (300, (1 << 30) // 3), (1 << 19, (1 << 19) - 128)]
EMBEDDING = [(1, 1, 1), (MANY, 1000, 512), (MANY, (1 << 29) - 1, 1), (1 << 24, 1000, 1 << 16),
             ((1 << 30) - 1, (1 << 29) - 1, 1024), ((1 << 30) - 1, 262144, 1024), (1, (1 << 29) - 1, 2048), (512, 200000, 512),
             (16384, 262145, 8)]
# [M][K] by [N][K]: up to 2^22 - 1 tiles of 128 x 128 in y, and either side of 2^28 columns for few rows
PRODUCTS = [(1, 1, 1), (1, (1 << 28) - 16, 128), (1, 1 << 28, 128), (4, 1 << 28, 128), (4, (1 << 28) + 5, 512), (5, 1 << 28, 1),
            (16, 1 << 28, 200), (1, (1 << 29) - 128, 128), ((1 << 29) - 128, 1, 128), (128, (1 << 29) - 128, 1),
            (1 << 18, (1 << 18) - 128, 1024), (300, 300, (1 << 23) - 128), (1, 4096, (1 << 23) - 128)]


@pytest.fixture(scope="module")
def calls(tmp_path_factory):
    if not shutil.which("gcc"):
        pytest.skip("no gcc")
    d = tmp_path_factory.mktemp("runtime")
    (d / "runtime.c").write_text(RUNTIME)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", str(d / "runtime.c"), "-o", str(d / "runtime.so")], check=True)
    r = subprocess.run([sys.executable, os.path.abspath(__file__), str(d / "runtime.so")], capture_output=True, text=True,
                       cwd=ROOT, timeout=300)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout.splitlines()[-1])


def test_every_launch_has_a_grid_that_the_runtime_takes(calls):
    for name, (status, launches) in calls.items():
        assert status == 0 and launches, name
        for blocks, threads in launches:
            assert 0 < threads <= 1024 and 0 < blocks < 1 << 31 and blocks * threads < 1 << 32, (name, blocks, threads)


def test_quantising_takes_every_tile_once(calls):
    for R, C in QUANTIZE:
        tiles = -(-R // 128) * -(-C // 128)
        assert tiles < 1 << 24
        for name, (_, launches) in calls.items():
            if name.startswith(f"quantize {R} {C} "):
                assert sum(blocks for blocks, _ in launches) == tiles, name


if __name__ == "__main__":
    run(sys.argv[1])
