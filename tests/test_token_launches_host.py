"""Host checks of the token operators' launches: a launch holds fewer than 2^32
threads, and none follows one that failed.  The runtime's launch functions are
replaced by ones that write down what they are given, so sizes up to the
documented limits are checked without a GPU and without their memory."""
import json
import os
import subprocess
import sys

import pytest

from conftest import ROOT
from dlrm_embedding_bag_amd import abi

RECORDER = r"""
#include <stddef.h>
#include <stdint.h>
typedef struct { uint32_t x, y, z; } dim3;
static dim3 grids[64], blocks[64], next_grid, next_block;
static int count, fail_at = -1, last;
void rec_reset(int fail) { count = 0; fail_at = fail; last = 0; }
int rec_count(void) { return count; }
uint64_t rec_threads(int i, int axis) {
  const uint32_t *g = &grids[i].x, *b = &blocks[i].x;
  return (uint64_t)g[axis] * b[axis];
}
uint32_t rec_block(int i) { return blocks[i].x * blocks[i].y * blocks[i].z; }
int __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, void *stream) {
  (void)lds; (void)stream;
  next_grid = grid;
  next_block = block;
  return 0;
}
int __hipPopCallConfiguration(dim3 *grid, dim3 *block, size_t *lds, void **stream) {
  *grid = next_grid;
  *block = next_block;
  *lds = 0;
  *stream = 0;
  return 0;
}
int hipLaunchKernel(const void *f, dim3 grid, dim3 block, void **args, size_t lds, void *stream) {
  (void)f; (void)args; (void)lds; (void)stream;
  if (count < 64) {
    grids[count] = grid;
    blocks[count] = block;
  }
  if (count++ == fail_at) last = 9;
  return last;
}
int hipGetLastError(void) {
  const int e = last;
  last = 0;
  return e;
}
"""

# Runs the calls given as JSON on stdin, [name, arguments, launch that fails or
# -1] each, and prints [status, [threads of the grid by axis, and of a
# workgroup, of each launch]].
DRIVER = r"""
import ctypes, json, sys
rec = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)   # found before the runtime's own
rec.rec_threads.restype = ctypes.c_uint64
sys.path.insert(0, sys.argv[2])
from dlrm_embedding_bag_amd import abi
lib = abi.load()
out = []
for name, args, fail in json.load(sys.stdin):
    rec.rec_reset(fail)
    status = getattr(lib, name)(*args)
    out.append([status, [[rec.rec_threads(i, a) for a in range(3)] + [rec.rec_block(i)]
                         for i in range(rec.rec_count())]])
print(json.dumps(out))
"""

FAKE = 0x10000  # never dereferenced: nothing is launched
F32, BF16, FP8 = 0, 1, 2
OK, HIP = 0, 5
INT32_MAX = 2**31 - 1


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    if not os.path.exists(abi.LIB_PATH):
        from dlrm_embedding_bag_amd import build
        build.build()
    folder = tmp_path_factory.mktemp("recorder")
    source, library = folder / "recorder.c", folder / "librecorder.so"
    source.write_text(RECORDER)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-o", str(library), str(source)], check=True)

    def run(calls):
        done = subprocess.run([sys.executable, "-c", DRIVER, str(library), ROOT],
                              input=json.dumps(calls), capture_output=True, text=True,
                              timeout=120)
        assert done.returncode == 0, done.stderr
        return json.loads(done.stdout)

    return run


def _grad(n, rows, dim, acc, ldo, gdt=BF16, odt=F32, fail=-1):
    return ["emb_lookup_grad", [n, rows, dim, FAKE, 0, gdt, FAKE, 1.0, acc, FAKE, ldo, odt, FAKE,
                                1 << 62, None], fail]


def _check(launches, calls):
    for call, (status, made) in zip(calls, launches(calls)):
        assert status == OK, call
        assert made, call
        for x, y, z, block in made:
            assert 0 < x < 2**32 and 0 < y < 2**32 and 0 < z < 2**32, (call, made)
            assert x * y * z < 2**32, (call, made)
            assert 0 < block <= 1024, (call, made)


def test_gradient_launches_hold_fewer_than_2_to_32_threads(launches):
    tokens = [0, 1, 1024, 1025, 2048, 2049, 65536, 65537, 2_500_000, 4_194_304, 4_194_305]
    tokens += [(1 << b) + d for b in range(23, 31) for d in (-1, 0, 1)] + [532_000_000, INT32_MAX]
    calls = []
    for n in tokens:
        for rows in (1, 100_000, INT32_MAX - 1):
            for dim in (1, 64, 520, 1 << 20):
                for acc, ldo in ((0, dim), (0, dim + 1), (1, dim)):
                    if n or not acc:
                        calls.append(_grad(n, rows, dim, acc, ldo))
    _check(launches, calls)


def test_gradient_stops_at_a_launch_that_failed(launches):
    """What follows reads what it should have written."""
    for n in (100, 5000, 100_000, 5_000_000):
        whole = _grad(n, 1000, 8, 0, 8)
        (status, made), = launches([whole])
        assert status == OK
        calls = [_grad(n, 1000, 8, 0, 8, fail=i) for i in range(len(made))]
        for i, (status, first) in enumerate(launches(calls)):
            assert status == HIP, (n, i)
            assert first == made[:i + 1], (n, i)


def test_other_launches_hold_fewer_than_2_to_32_threads(launches):
    calls = []
    for n in (1, 1000, 1 << 20, (1 << 28) + 1, INT32_MAX):
        for dim in (1, 5, 64, 1024, 1 << 20):
            for table, out in ((F32, F32), (BF16, BF16), (FP8, BF16)):
                calls.append(["emb_lookup_scaled", [n, 1000, dim, FAKE, dim, table, FAKE, 1.0,
                                                    FAKE, dim, out, None], -1])
    for m in (1, 512, 513, 1 << 20, 1 << 32, 1 << 36):
        for dim in (1, 33, 64, 65, 129, 512, 1024, 2048, 4096, 8192, 8193, 1 << 20):
            calls.append(["rms_norm_residual_i8", [m, dim, FAKE, 0, FAKE, 0, BF16, FAKE, 1e-6, FAKE,
                                                   dim, FAKE, dim, FAKE, None], -1])
    # outputs of up to 2^38 elements
    for m in (1, 16, 64, 65, 4096, 1 << 20, 1 << 26):
        for n in (1, 16, 8192, 1 << 20, 1 << 26):
            for k in (1, 415, 4096):
                if m * n <= 1 << 38:
                    calls.append(["linear_i8_bias_act", [m, n, k, FAKE, k, FAKE, FAKE, k, FAKE,
                                                         None, 0, FAKE, n, BF16, None], -1])
    _check(launches, calls)


def test_gradient_takes_one_launch_up_to_2048_tokens(launches):
    """and one merge up to 32 tiles of 2048; the workspace begins with the tiles."""
    def made(n):
        (status, all_launches), = launches([_grad(n, 1000, 8, 0, 8)])
        assert status == OK
        return len(all_launches)

    bytes_of = abi.load().emb_lookup_grad_workspace_bytes
    assert made(2048) == 1 and bytes_of(2048, 1000, 8) == 0
    assert made(2049) == 4 and bytes_of(2049, 1000, 8) > 0      # sort, merge, reduce, fix
    assert made(65536) == 4
    assert made(65537) == 5
    assert made(2_500_001) == 6                                 # three merges
