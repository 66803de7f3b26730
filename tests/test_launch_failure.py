"""A launch that the runtime refuses: status, and what the call leaves behind.
The CUDA runtime is a fake here (no GPU needed): it answers the library's
queries as a GB300 would, refuses the launch it is told to, and writes down
every launch and memset."""
import json
import os
import shutil
import subprocess
import sys

import pytest

import token_sampling_logits_gb300 as gs

FAKE = r"""
#include <stddef.h>
static int refused = -1, launches = 0, memsets = 0;
static void* memset_at = 0;
static size_t memset_bytes = 0;
static int memset_value = -1, memset_after = 0;
void fake_refuse(int nth) { refused = nth; launches = memsets = 0; }
int fake_launches(void) { return launches; }
int fake_memsets(void) { return memsets; }
void* fake_memset_at(void) { return memset_at; }
size_t fake_memset_bytes(void) { return memset_bytes; }
int fake_memset_value(void) { return memset_value; }
int fake_memset_after(void) { return memset_after; }

int cudaGetDevice(int* d) { *d = 0; return 0; }
int cudaGetLastError(void) { return 0; }
int cudaDeviceGetAttribute(int* v, int attr, int dev) {
  (void)dev;
  *v = attr == 75 ? 10 : attr == 76 ? 3 : attr == 16 ? 152 : 0;  /* major, minor, SMs */
  return 0;
}
int cudaFuncSetAttribute(const void* f, int a, int v) { (void)f; (void)a; (void)v; return 0; }
int cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void* f, int b, size_t s,
                                                           unsigned g) {
  (void)f; (void)b; (void)s; (void)g;
  *n = 2;
  return 0;
}
int cudaOccupancyMaxActiveClusters(int* n, const void* f, const void* c) {
  (void)f; (void)c;
  *n = 16;
  return 0;
}
int cudaOccupancyMaxPotentialClusterSize(int* n, const void* f, const void* c) {
  (void)f; (void)c;
  *n = 8;
  return 0;
}
int cudaLaunchKernelExC(const void* cfg, const void* f, void** args) {
  (void)cfg; (void)f; (void)args;
  return launches++ == refused ? 1 : 0;
}
int cudaMemsetAsync(void* p, int v, size_t n, void* stream) {
  (void)stream;
  ++memsets;
  memset_at = p; memset_bytes = n; memset_value = v; memset_after = launches;
  return 0;
}
"""

CHILD = r"""
import ctypes, json, sys
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)  # found before the real runtime
fake.fake_memset_at.restype = ctypes.c_void_p
fake.fake_memset_bytes.restype = ctypes.c_size_t
import token_sampling_logits_gb300 as gs
L, AT = gs.lib(), 1 << 30
B, V = int(sys.argv[2]), 50000
s = gs._StateC(AT, AT, AT, B, V, 50016)
c = gs._ConstraintsC()
c.state = ctypes.addressof(s)
out = []
for nth in (-1, 0, 1):
    fake.fake_refuse(nth)
    st = L.gsample_constrained_gumbel_argmax(AT, gs.BF16, B, V, V, AT, AT, AT, ctypes.byref(c), AT,
                                             3 * AT, None)
    out.append(dict(refused=nth, status=st, launches=fake.fake_launches(),
                    memsets=fake.fake_memsets(), at=fake.fake_memset_at(),
                    bytes=fake.fake_memset_bytes(), value=fake.fake_memset_value(),
                    after=fake.fake_memset_after()))
print(json.dumps(out))
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    if not shutil.which("gcc"):
        pytest.skip("needs gcc")
    at = tmp_path_factory.mktemp("fake")
    (at / "fake.c").write_text(FAKE)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(at / "libfake.so"), str(at / "fake.c")],
                   check=True)
    return str(at / "libfake.so")


def calls(fake, B):
    gs.lib()  # built
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CHILD, fake, str(B)], cwd=root, check=True,
                       capture_output=True, text=True, timeout=120)
    return json.loads(r.stdout)


def test_a_constrained_draw_whose_second_launch_is_refused_leaves_a_clean_workspace(fake):
    """The first launch publishes scores in the workspace, which the second one
    would have cleared."""
    both, first, second = calls(fake, 256)
    assert (both["status"], both["launches"], both["memsets"]) == (gs.OK, 2, 0)
    assert (first["status"], first["launches"], first["memsets"]) == (gs.ERR_CUDA, 1, 0)
    assert (second["status"], second["launches"]) == (gs.ERR_CUDA, 2)
    assert second["memsets"] == 1 and second["after"] == 2
    assert (second["at"], second["value"], second["bytes"]) == (3 << 30, 0, gs.workspace_bytes(256))


def test_a_small_batch_takes_one_launch_and_no_workspace(fake):
    one, refused, _ = calls(fake, 4)
    assert (one["status"], one["launches"], one["memsets"]) == (gs.OK, 1, 0)
    assert (refused["status"], refused["launches"], refused["memsets"]) == (gs.ERR_CUDA, 1, 0)
