"""The library's host code with the CUDA runtime and the kernels' launches replaced.

The objects of the API's sources are linked with functions of the same names
that note on which device they were called: two devices, no GPU.
"""
import ctypes
import os
import shutil
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "model_free_suffix_gb300")

SOURCE = r"""
#include <stdlib.h>
#include <string.h>
#include <string>
#include <cuda_runtime_api.h>
#include "verify.h"

static thread_local int current = 0;   // (as the runtime keeps it)
static thread_local std::string seen;
extern "C" void fake_note(const char *name) { seen += name; seen += "@"; seen += std::to_string(current); seen += "\n"; }
extern "C" const char *fake_seen() { static std::string out; out = seen; seen.clear(); return out.c_str(); }
extern "C" void fake_set(int d) { current = d; }
extern "C" int fake_get() { return current; }

extern "C" cudaError_t cudaGetDevice(int *d) { *d = current; return cudaSuccess; }
extern "C" cudaError_t cudaSetDevice(int d) {
  if (d < 0 || d > 1) return cudaErrorInvalidDevice;
  current = d;
  return cudaSuccess;
}
extern "C" cudaError_t cudaMalloc(void **p, size_t n) { fake_note("cudaMalloc"); *p = calloc(1, n + 256); return cudaSuccess; }
extern "C" cudaError_t cudaFree(void *p) { fake_note("cudaFree"); free(p); return cudaSuccess; }
extern "C" cudaError_t cudaMallocHost(void **p, size_t n) { *p = calloc(1, n + 256); return cudaSuccess; }
extern "C" cudaError_t cudaFreeHost(void *p) { free(p); return cudaSuccess; }
extern "C" cudaError_t cudaMemcpy(void *to, const void *from, size_t n, cudaMemcpyKind) {
  fake_note("cudaMemcpy");
  memcpy(to, from, n);
  return cudaSuccess;
}
extern "C" cudaError_t cudaMemset(void *to, int c, size_t n) { memset(to, c, n); return cudaSuccess; }
namespace sgd {
VerifyLayout verify_layout(int, int) { return VerifyLayout{0, 0, 4096}; }
}
"""


def build(folder) -> ctypes.CDLL:
    from model_free_suffix_gb300 import build as B
    B.build()
    objects = [os.path.join(B.OUT_DIR, f) for f in ("api.cu.o", "kv_api.cu.o")]
    cuda = os.path.join(os.path.dirname(os.path.dirname(shutil.which("nvcc") or B.nvcc())), "include")
    source = os.path.join(str(folder), "fake.cpp")
    flags = ["g++", "-std=c++17", "-O1", "-fPIC", "-I", cuda, "-I", os.path.join(PACKAGE, "csrc")]

    def names(path, *options):
        out = subprocess.check_output(["nm", *options, path], text=True)
        return {line.split()[-1] for line in out.splitlines() if line.strip()}

    with open(source, "w") as f:
        f.write(SOURCE)
    first = os.path.join(str(folder), "fake.o")
    subprocess.check_call(flags + ["-c", source, "-o", first])
    have = names(first, "--defined-only", "-g").union(*(names(o, "--defined-only", "-g") for o in objects))
    need = sorted(n for o in objects for n in names(o, "-u")
                  if n not in have and (n.startswith(("cuda", "__cuda")) or n.startswith("_ZN3sgd")))
    stubs = os.path.join(str(folder), "stubs.cpp")
    with open(stubs, "w") as f:
        f.write('extern "C" void fake_note(const char *);\n')
        for i, n in enumerate(dict.fromkeys(need)):
            f.write('extern "C" long stub%d() __asm__("%s");\n' % (i, n))
            quiet = n.startswith("__cuda")
            f.write('extern "C" long stub%d() { %sreturn 0; }\n' % (i, "" if quiet else 'fake_note("%s"); ' % n))
    out = os.path.join(str(folder), "libfake.so")
    # (its own functions first, whatever else the process has loaded)
    subprocess.check_call(flags + ["-shared", "-Wl,-Bsymbolic", "-o", out, first, stubs] + objects + ["-lpthread"])
    return ctypes.CDLL(out)
