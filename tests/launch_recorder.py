"""Launches of the dense block's entry points without a GPU: the HIP calls of
libfff.so go to stand-ins that note each launch (kernel, workgroups, threads)
and refuse what HIP refuses.  The stand-ins must come before HIP, so the calls
are made in a process of their own: record() starts it, and this file is its
program.  Pointers are never followed."""
import ctypes
import json
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STAND_INS = r"""
#include <cstddef>
#include <cstdint>
#include <cstring>
#include <map>
#include <string>
#include <vector>
struct Dim { uint32_t x, y, z; };
struct Launch { const char* name; Dim grid, block; };
static std::map<const void*, std::string>& names() { static std::map<const void*, std::string> m; return m; }
static std::vector<Launch> launches;
static struct { Dim grid, block; size_t lds; void* stream; } config;
static int last = 0, capturing = 0;
extern "C" {
void** __hipRegisterFatBinary(const void*) { static void* handle; return &handle; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*,
                           int*) { names()[host] = name; }
int __hipPushCallConfiguration(Dim grid, Dim block, size_t lds, void* stream) {
  config = {grid, block, lds, stream};
  return 0;
}
int __hipPopCallConfiguration(Dim* grid, Dim* block, size_t* lds, void** stream) {
  *grid = config.grid, *block = config.block, *lds = config.lds, *stream = config.stream;
  return 0;
}
int hipLaunchKernel(const void* host, Dim grid, Dim block, void**, size_t lds, void*) {
  const uint64_t threads = uint64_t(grid.x) * block.x;
  // (invalid configuration: nothing to run, or more than a launch has)
  if (!grid.x || !grid.y || !grid.z || !block.x || block.x > 1024 || threads >> 32 || lds > 160 * 1024) return last = 9;
  launches.push_back({names()[host].c_str(), grid, block});
  return 0;
}
int hipGetLastError() { const int e = last; last = 0; return e; }
int hipGetDevice(int* d) { *d = 0; return 0; }
int hipFuncSetAttribute(const void*, int, int) { return 0; }
int hipStreamIsCapturing(void*, int* status) { *status = capturing; return 0; }
void record_start(int capture) { launches.clear(); last = 0; capturing = capture; }
int record_count() { return int(launches.size()); }
const char* record_get(int i, uint32_t* grid, uint32_t* block) {
  *grid = launches[i].grid.x, *block = launches[i].block.x;
  return launches[i].name;
}
}
"""

# Pointer arguments of the entry points, in their order.
ARGS = {
    "fff_linear": ["x", "W", "bias", "residual", "y", "pre", "pre_scale", "ws"],
    "fff_linear_backward": ["dy", "x", "x_scale", "W", "pre", "pre_scale", "dx", "dW", "dbias", "ws"],
    "fff_gated": ["x", "Wg", "Wu", "h", "gate", "gate_scale", "up", "up_scale", "ws"],
    "fff_gated_backward": ["dh", "x", "x_scale", "Wg", "Wu", "gate", "gate_scale", "up", "up_scale", "dx",
                           "dWg", "dWu", "h", "ws"],
}


def build(where):
    """The stand-ins, compiled into the folder `where`."""
    src, lib = os.path.join(where, "stand_ins.cpp"), os.path.join(where, "stand_ins.so")
    with open(src, "w") as f:
        f.write(STAND_INS)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-w", src, "-o", lib], check=True)
    return lib


def record(lib, calls):
    """calls: [(entry point, shape's fields, pointers other than the default by
    name, capturing)].  Returns [(status, [(kernel, workgroups, threads)])]."""
    r = subprocess.run([sys.executable, os.path.abspath(__file__), lib], input=json.dumps(calls), text=True,
                       capture_output=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return [(status, [tuple(k) for k in kernels]) for status, kernels in json.loads(r.stdout)]


def main():
    sys.path.insert(0, ROOT)
    stand_ins = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
    stand_ins.record_get.restype = ctypes.c_char_p
    import sparse_tree_structured_amd as fff
    lib = fff.load_library()
    grid, block, out = ctypes.c_uint32(), ctypes.c_uint32(), []
    for name, fields, pointers, capturing in json.load(sys.stdin):
        stand_ins.record_start(int(capturing))
        p = [pointers.get(k, 1 << 40) for k in ARGS[name]]
        status = getattr(lib, name)(fff.DenseShape(**fields), *p, 1 << 62, None)
        kernels = [(stand_ins.record_get(i, ctypes.byref(grid), ctypes.byref(block)).decode(), grid.value, block.value)
                   for i in range(stand_ins.record_count())]
        out.append((status, kernels))
    json.dump(out, sys.stdout)


if __name__ == "__main__":
    main()
