"""Launches that fail, without a GPU: the library's host code runs in a child process against a fake
of the CUDA runtime's calls, whose launches return an error code every time or once."""
import os
import subprocess
import sys

import pytest

FAKE = r"""
#include <cuda.h>
#include <cuda_runtime_api.h>
#include <stdlib.h>
#include <string.h>

static int launches, refused, limit, last = cudaSuccess, failing;
static void (*on_limit)(void);
int fake_launches(void) { return launches; }
int fake_refused(void) { return refused; }
int fake_last(void) { return last; }
/* called once, right behind the next change of a limit */
void fake_on_limit(void (*f)(void)) { on_limit = f; }
/* the next n launches fail with cudaErrorInvalidValue, and one that wants more dynamic shared
   memory than the kernel's limit always does */
void fake_reset(int n) { launches = refused = 0; last = cudaSuccess; failing = n; }
void fake_leave_error(int e) { last = e; }

cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr a, int d) { *v = 152; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void* f, enum cudaFuncAttribute a, int v) {
  void (*then)(void) = on_limit;
  limit = v;
  on_limit = 0;
  if (then) then();
  return cudaSuccess;
}
cudaError_t cudaFuncGetAttributes(struct cudaFuncAttributes* a, const void* f) {
  memset(a, 0, sizeof *a);
  a->numRegs = 128;
  return cudaSuccess;
}
cudaError_t cudaGetLastError(void) { cudaError_t e = (cudaError_t)last; last = cudaSuccess; return e; }
static cudaError_t launch(size_t smem) {
  ++launches;
  if ((failing <= 0 || failing-- == 0) && (smem <= 48 * 1024 || smem <= (size_t)limit)) return cudaSuccess;
  ++refused;
  last = cudaErrorInvalidValue;
  return cudaErrorInvalidValue;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
  return launch(c->dynamicSmemBytes);
}
cudaError_t cudaLaunchKernel(const void* f, dim3 g, dim3 b, void** args, size_t smem, cudaStream_t s) {
  return launch(smem);
}
cudaError_t __cudaLaunchKernel(cudaKernel_t f, dim3 g, dim3 b, void** args, size_t smem, cudaStream_t s) {
  return launch(smem);
}
static CUresult encode(void) { return CUDA_SUCCESS; }
cudaError_t cudaGetDriverEntryPointByVersion(const char* n, void** p, unsigned int v, unsigned long long f,
                                             enum cudaDriverEntryPointQueryResult* q) {
  *p = (void*)encode;
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
"""

CHILD = r"""
import ctypes, sys
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)   # found before the runtime's own symbols
lib = ctypes.CDLL(sys.argv[2])
P, I, L, Z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
lib.msa_build_page_tables.argtypes = [P, P, I, I, P, P, I, P, P, I, L, I, P, P, P, P, P, P]
lib.msa_append_kv.argtypes = [P, L, P, L, P, L, P, I, I, I, I, L, P, P, P, P]
lib.msa_shared_prefix_decode.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, L, P, P, P, Z, P]
at = [0x1000000 * (i + 1) for i in range(20)]                # device pointers, never dereferenced

def tables(B):
    return lib.msa_build_page_tables(at[0], at[1], B, 8, at[2], at[3], 10, at[4], None, 0, 64, 16, at[5],
                                     at[6], at[7], at[8], at[9], None)

def append():
    return lib.msa_append_kv(at[0], 1024, at[1], 1024, at[2], 1024, at[3], 4, 8, 128, 128, 16, at[4], at[5],
                             at[6], None)

def decode():
    return lib.msa_shared_prefix_decode(at[0], at[1], at[2], at[3], at[4], at[5], 4, 1, 64, 8, 128, 16, 64,
                                        at[6], at[7], at[8], 1 << 30, None)

exec(sys.argv[3])
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    from block_sparse_attention_msa_gb300 import build
    lib = build.build()
    d = tmp_path_factory.mktemp("fake")
    src, so = d / "fake.c", d / "fake.so"
    src.write_text(FAKE)
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc()))), "include")
    subprocess.run(["gcc", "-shared", "-fPIC", "-w", "-I", include, str(src), "-o", str(so)], check=True)

    def go(code):
        r = subprocess.run([sys.executable, "-c", CHILD, str(so), lib, code], capture_output=True, text=True,
                           timeout=120)
        assert r.returncode == 0, f"exit {r.returncode}\n{r.stderr[-2000:]}"

    return go


def test_the_fake_is_the_one_that_is_called(run):
    run("for call, n in ((lambda: tables(4), 1), (append, 1), (decode, 2)):\n"
        "    fake.fake_reset(0)\n"
        "    assert call() == 0 and fake.fake_launches() == n, fake.fake_launches()")


@pytest.mark.parametrize("call", ["tables(7000)", "tables(16384)", "tables(4)", "append()", "decode()"])
def test_a_launch_that_keeps_failing_is_an_error(run, call):
    # -5: MSA_ERR_CUDA. At most one more attempt, and no error left behind for the thread's next call.
    run(f"fake.fake_reset(1 << 30)\nassert {call} == -5 and 1 <= fake.fake_launches() <= 2, fake.fake_launches()\n"
        "assert fake.fake_last() == 0\n"
        f"fake.fake_reset(0)\nassert {call} == 0")


def test_a_launch_that_fails_once_is_made_again(run):
    # as after a device reset, which drops the limit that the library raised
    run("fake.fake_reset(0)\nassert tables(7000) == 0\n"
        "fake.fake_reset(1)\nassert tables(7000) == 0 and fake.fake_launches() == 2 and fake.fake_last() == 0")


def test_two_batch_sizes_at_once_do_not_lower_each_others_limit(run):
    # the small batch runs whole between the large one's raise of the limit and its launch
    run("fake.fake_reset(0)\ninner = []\n"
        "cb = ctypes.CFUNCTYPE(None)(lambda: inner.append(tables(7000)))\n"
        "fake.fake_on_limit(cb)\n"
        "assert tables(16384) == 0 and inner == [0]\n"
        "assert fake.fake_refused() == 0 and fake.fake_launches() == 2")


@pytest.mark.parametrize("call", ["tables(4)", "append()", "decode()"])
def test_an_older_error_of_the_thread_is_not_the_calls(run, call):
    # 1: cudaErrorInvalidValue of some earlier call, not yet read; it stays for whoever reads it
    run(f"fake.fake_reset(0)\nfake.fake_leave_error(1)\nassert {call} == 0 and fake.fake_last() == 1")


def test_neighbouring_buffers_do_not_overlap(run):
    # 4 lengths, 10 free pages, 16 rows and a table of 4 x 8 in one allocation, end to end; an empty
    # buffer overlaps nothing
    run("""fake.fake_reset(0)
def call(free, nfree, T, slots, pos):
    return lib.msa_build_page_tables(0x10000, 0x10010, 4, 8, 0x20000, free, nfree, 0x10020, None, 0, 64, T,
                                     0x10024, 0x10034, slots, pos, 0x10048, None)
assert call(0x1004c, 10, 16, 0x10074, 0x100b4) == 0
assert call(0x10028, 0, 0, 0x20004, 0x20004) == 0
assert call(0x1004c, 10, 16, 0x10074, 0x100b0) == -1""")
