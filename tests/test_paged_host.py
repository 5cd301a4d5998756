"""The host side of include/paged.h over a stand-in for the CUDA runtime (a
library that is loaded ahead of it): several devices, and what happens between
two operations of a call.  No GPU."""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A kernel that wants more than 48 KB of shared memory launches only on a device
# where its attribute was set to as much.  Memory of the device is host memory.
FAKE = r"""
#include <stddef.h>
#include <stdint.h>
#include <string.h>
typedef struct { unsigned grid[3], block[3]; size_t smem; void* stream; void* attrs; unsigned n; } Config;
int fake_device = 0, fake_launches = 0, fake_word = 0, fake_or_after_read = 0, fake_fail_attribute = 0;
static struct { const void* f; int dev, bytes; } set[256];
static int sets = 0;
int cudaGetDevice(int* d) { *d = fake_device; return 0; }
int cudaDeviceGetAttribute(int* v, int a, int d) { (void)a; (void)d; *v = 152; return 0; }
int cudaGetSymbolAddress(void** p, const void* s) { (void)s; *p = &fake_word; return 0; }
int cudaGetDriverEntryPointByVersion(const char* n, void** f, unsigned v, unsigned long long g, void* q) {
  (void)n; (void)v; (void)g; (void)q; *f = 0; return 1;
}
int cudaFuncSetAttribute(const void* f, int a, int bytes) {
  (void)a;
  if (fake_fail_attribute) { --fake_fail_attribute; return 46; }
  set[sets].f = f; set[sets].dev = fake_device; set[sets].bytes = bytes;
  ++sets;
  return 0;
}
int cudaLaunchKernelExC(const Config* c, const void* f, void** args) {
  (void)args;
  int most = 48 * 1024;
  for (int i = 0; i < sets; ++i)
    if (set[i].f == f && set[i].dev == fake_device) most = set[i].bytes;
  if (c->smem > (size_t)most) return 1;  // cudaErrorInvalidValue
  ++fake_launches;
  /* the kernel that takes bits out of the error word: (int* word, int bits) */
  if (c->grid[0] == 1 && c->block[0] == 1 && *(int**)args[0] == &fake_word)
    fake_word &= ~*(int*)args[1];
  return 0;
}
int cudaMemcpyAsync(void* d, const void* s, size_t n, int k, void* st) {
  (void)k; (void)st;
  memcpy(d, s, n);
  if (s == &fake_word) fake_word |= fake_or_after_read;  /* a kernel of another stream */
  return 0;
}
int cudaMemsetAsync(void* d, int v, size_t n, void* st) { (void)st; memset(d, v, n); return 0; }
int cudaStreamSynchronize(void* st) { (void)st; return 0; }
"""

CHILD = r"""
import ctypes, json, sys
fake = ctypes.CDLL(sys.argv[1])
lib = ctypes.CDLL(sys.argv[2])
class Cache(ctypes.Structure):
    _fields_ = [(n, t) for t, ns in ((ctypes.c_void_p, "k v"), (ctypes.c_int, "dtype pages page heads dim"),
                                     (ctypes.c_int64, "ps rs hs")) for n in ns.split()]
class Batch(ctypes.Structure):
    _fields_ = [(n, t) for t, ns in ((ctypes.c_void_p, "table cu kv"), (ctypes.c_int, "N T width"),
                                     (ctypes.c_int64, "ts")) for n in ns.split()]
A = 0x10000
L, P = ctypes.c_int64, ctypes.c_void_p
def var(name):
    return ctypes.c_int.in_dll(fake, name)
def attend(dim, T, dtype=1, page=16):
    c = Cache(A, A, dtype, 64, page, 2, dim, page * 2 * dim, 2 * dim, dim)
    b = Batch(A, A, A, 1, T, 8, 8)
    n = ctypes.c_size_t()
    assert lib.paged_attention_workspace(ctypes.byref(c), ctypes.byref(b), 4, 0, T, 100, ctypes.byref(n)) == 0
    return lib.paged_attention(P(A), L(4 * dim), L(dim), 4, ctypes.byref(c), ctypes.byref(b), ctypes.c_float(0.1),
                               1, 0, T, 100, P(A), L(4 * dim), L(dim), None, P(A), n, None)
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    from sparse_moe_bit_gb300 import build, moe
    if not os.path.exists(moe.LIB_PATH):
        build.build()
    d = tmp_path_factory.mktemp("fake")
    src, so = d / "fake.c", d / "fake.so"
    src.write_text(FAKE)
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", str(so), str(src)], check=True)

    def call(code):
        env = dict(os.environ, LD_PRELOAD=str(so))
        r = subprocess.run([sys.executable, "-c", CHILD + code, str(so), moe.LIB_PATH], env=env,
                           capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr
        return json.loads(r.stdout.splitlines()[-1])
    return call


def test_every_device_gets_its_kernels_shared_memory(run):
    """The first call on a second device of the process: each variant (rows and
    chunk, every head size, both types)."""
    r = run(r"""
out = []
for dim in (64, 128, 256):
    for T in (1, 8, 40):
        for dtype in (1, 2):
            for dev in (0, 1, 0, 63, 1):
                var("fake_device").value = dev
                out.append(attend(dim, T, dtype))
print(json.dumps([out, var("fake_launches").value]))
""")
    assert r[0] == [0] * len(r[0]) and r[1] >= len(r[0])


def test_a_failed_attribute_is_set_again(run):
    r = run(r"""
var("fake_fail_attribute").value = 1
print(json.dumps([attend(128, 1), attend(128, 1)]))
""")
    assert r[0] == 3 and r[1] == 0


def test_error_bits_set_while_the_word_is_read_are_not_lost(run):
    """A kernel on another stream sets a bit between the read of the error word and
    its clearing: the next call reports it."""
    r = run(r"""
code = ctypes.c_int()
out = []
var("fake_word").value = 2
var("fake_or_after_read").value = 1
for i in range(3):
    out.append([lib.paged_get_device_error(None, ctypes.byref(code)), code.value])
    var("fake_or_after_read").value = 0
print(json.dumps(out))
""")
    assert r == [[5, 2], [5, 1], [0, 0]]


def test_a_batch_of_single_tokens_takes_the_kernel_for_few_rows_unasked(run):
    """Without max_q the mean number of new tokens chooses: a decode batch gets the
    plan that max_q = 1 gets, more than 8 rows a key/value head (4 query heads each
    here) the plan of chunks."""
    r = run(r"""
def size(N, T, max_q, max_kv=0):
    c = Cache(A, A, 1, 4096, 16, 2, 128, 16 * 256, 256, 128)
    b = Batch(A, A, A, N, T, 256, 256)
    n = ctypes.c_size_t()
    assert lib.paged_attention_workspace(ctypes.byref(c), ctypes.byref(b), 8, 0, max_q, max_kv,
                                         ctypes.byref(n)) == 0
    return n.value
few = [[size(64, 64, 0), size(64, 64, 1), size(64, 64, 64)],
       [size(64, 128, 0), size(64, 128, 2), size(64, 128, 65)]]
many = [[size(8, 24, 0), size(8, 24, 17), size(8, 24, 3)],
        [size(8, 800, 0), size(8, 800, 100), size(8, 800, 1)]]
print(json.dumps([few, many, size(0, 0, 0), size(0, 5, 0)]))
""")
    for none, mean, other in r[0] + r[1]:
        assert none == mean and none != other
