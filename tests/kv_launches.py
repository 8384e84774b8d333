"""What an entry point launches, without a GPU: a stand-in for the HIP runtime takes every call of the host code and
records the launches. It answers as a runtime with one gfx950 does; a launch of 2^32 threads or more fails, as there.

recorded(calls) runs each call (entry point, its arguments) in a process of its own, in which nothing else has loaded the
runtime, and returns (return code, launches) of each. An argument is a number, None, a float or bytes (a structure of the
header, passed by address). A launch is a dict: kernel, grid, block, q (address, row stride in bytes and rows, the first
three words of the kernel's first argument), and `more` (the next two arguments of kv_write_kernel).
"""
import ctypes
import json
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <hip/hip_runtime_api.h>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <map>
#include <string>

static std::map<const void*, std::string> names;
static std::string record;
static dim3 grid_, block_;
static int symbol;

extern "C" {
void** __hipRegisterFatBinary(const void*) { static void* handle; return &handle; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* f, char*, const char* name, unsigned, uint3*, uint3*, dim3*, dim3*, int*) { names[f] = name; }
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, hipStream_t) {
  grid_ = grid;
  block_ = block;
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* st) {
  *grid = grid_;
  *block = block_;
  *lds = 0;
  *st = nullptr;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t, hipStream_t) {
  const std::string& name = names[f];
  int64_t q[3];
  std::memcpy(q, args[0], sizeof(q));
  int more[2] = {0, 0};
  if (name.find("kv_write_kernel") != std::string::npos)
    for (int i = 0; i < 2; ++i) more[i] = *static_cast<int*>(args[1 + i]);
  char line[512];
  std::snprintf(line, sizeof(line), "{\"kernel\": \"%.200s\", \"grid\": %u, \"block\": %u, \"q\": [%lld, %lld, %lld], \"more\": [%d, %d]}",
                name.c_str(), grid.x, block.x, (long long)q[0], (long long)q[1], (long long)q[2], more[0], more[1]);
  record += (record.empty() ? "" : ", ") + std::string(line);
  return static_cast<uint64_t>(grid.x) * block.x >> 32 ? hipErrorInvalidConfiguration : hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipGetDevice(int* dev) { *dev = 0; return hipSuccess; }
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipStreamGetDevice(hipStream_t, hipDevice_t* dev) { *dev = 0; return hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* s) { *s = hipStreamCaptureStatusNone; return hipSuccess; }
hipError_t hipGetDeviceProperties(hipDeviceProp_t* p, int) {
  std::memset(p, 0, sizeof(*p));
  std::strcpy(p->gcnArchName, "gfx950");
  p->multiProcessorCount = 256;
  return hipSuccess;
}
hipError_t hipPointerGetAttributes(hipPointerAttribute_t* a, const void*) {
  std::memset(a, 0, sizeof(*a));
  a->type = hipMemoryTypeDevice;
  return hipSuccess;
}
hipError_t hipDeviceGetDefaultMemPool(hipMemPool_t*, int) { return hipErrorNotSupported; }
hipError_t hipGetSymbolAddress(void** p, const void*) { *p = &symbol; return hipSuccess; }

const char* taken() {   // what was recorded since the last call of it
  static std::string last;
  last = "[" + record + "]";
  record.clear();
  return last.c_str();
}
}
"""


def recorded(calls, where):
    """(return code, launches) of every call; the stand-in is built in `where`."""
    from fp4_mqa_scoring_amd import build
    if not os.path.exists(build.LIB):
        build.build()
    src, lib = os.path.join(str(where), "runtime.hip"), os.path.join(str(where), "runtime.so")
    if not os.path.exists(lib):
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run([build.hipcc(), *build.HIPCC_FLAGS, "-w", src, "-o", lib], check=True, capture_output=True)
    sent = [[name, [dict(bytes=a.hex()) if isinstance(a, bytes) else a for a in args]] for name, args in calls]
    r = subprocess.run([sys.executable, os.path.abspath(__file__), lib, build.LIB], input=json.dumps(sent), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    return [(rc, launches) for rc, launches in json.loads(r.stdout)]


def main():
    runtime = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)     # found before the library's own
    runtime.taken.restype = ctypes.c_char_p
    lib = ctypes.CDLL(sys.argv[2])
    got = []
    for name, args in json.load(sys.stdin):
        kept, made = [], []
        for a in args:
            if isinstance(a, dict):
                kept.append(ctypes.create_string_buffer(bytes.fromhex(a["bytes"])))
                made.append(ctypes.cast(kept[-1], ctypes.c_void_p))
            else:
                made.append(a if a is None else ctypes.c_float(a) if isinstance(a, float) else ctypes.c_int64(a))
        rc = getattr(lib, name)(*made)
        got.append((rc, json.loads(runtime.taken())))
    json.dump(got, sys.stdout)


if __name__ == "__main__":
    main()
