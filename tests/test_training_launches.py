"""How the training operators' kernels are launched, without a GPU: the runtime's launch calls are replaced by ones that
write down what they are given."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

RECORDER = r"""
#include <stdio.h>
#include <stddef.h>
typedef struct { unsigned x, y, z; } dim3_t;
int hipFuncSetAttribute(const void *f, int attribute, int value) {
    printf("attribute %p %d %d\n", f, attribute, value);
    fflush(stdout);
    return 0;
}
int hipLaunchKernel(const void *f, dim3_t grid, dim3_t block, void **args, size_t lds, void *stream) {
    (void)args; (void)stream;
    printf("launch %p %u %u %u %u %zu\n", f, grid.x, grid.y, grid.z, block.x * block.y * block.z, lds);
    fflush(stdout);
    return 0;
}
static struct { dim3_t grid, block; size_t lds; void *stream; } held;
int __hipPushCallConfiguration(dim3_t grid, dim3_t block, size_t lds, void *stream) {
    held.grid = grid; held.block = block; held.lds = lds; held.stream = stream;
    return 0;
}
int __hipPopCallConfiguration(dim3_t *grid, dim3_t *block, size_t *lds, void **stream) {
    *grid = held.grid; *block = held.block; *lds = held.lds; *stream = held.stream;
    return 0;
}
int hipGetLastError(void) { return 0; }
int hipPeekAtLastError(void) { return 0; }
"""


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    from tile_binned_gaussian_amd import build
    if build.stale():
        build.build()
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    at = tmp_path_factory.mktemp("recorder")
    (at / "recorder.c").write_text(RECORDER)
    subprocess.run([gcc, "-shared", "-fPIC", "-o", str(at / "recorder.so"), str(at / "recorder.c")], check=True)
    return str(at / "recorder.so")


def recorded(recorder, calls):
    """The lines of a process that makes these calls of the library; its pointers are never dereferenced."""
    code = ("import ctypes\nfrom tile_binned_gaussian_amd import binding\nlib = binding.load_library()\n"
            "at = lambda k: ctypes.c_void_p(k << 40)\n" + calls)
    env = dict(os.environ, LD_PRELOAD=recorder, PYTHONPATH=ROOT)
    out = subprocess.run([sys.executable, "-c", code], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    return [line.split() for line in out.stdout.splitlines() if line.startswith(("attribute", "launch"))]


def test_a_kernels_largest_lds_size_is_one_value(recorder):
    """The attribute belongs to the kernel, not to a call: set to a call's own size, one thread's setting would be lowered
    by another's between its setting and its launch. So every call of a kernel sets the same, and none launches more."""
    lines = recorded(recorder, """
for experts in (8, 900, 1000, 1024, 1025, 3000, 4096):
    assert lib.gs_expert_plan(at(1), 64, 2, experts, at(2), at(3), at(4), None, 0, None) == 0
for m, n in ((96, 160), (128, 128), (32, 1000), (128, 96)):
    assert lib.gs_orthogonalize(at(1), 1, m, n, 5, 1.5, -0.5, 0.0, 1e-7, 0, at(2), None, 0, None) == 0
""")
    largest = {}
    for line in lines:
        if line[0] == "attribute":
            largest.setdefault(line[1], set()).add(int(line[3]))
        elif int(line[6]) + 1024 > 65536:
            assert line[1] in largest and int(line[6]) <= max(largest[line[1]])
    assert sum(line[0] == "launch" for line in lines) == 11
    assert len(largest) >= 2, "no kernel here needs more than 64 KB"
    assert all(len(sizes) == 1 for sizes in largest.values()), largest
