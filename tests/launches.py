"""Which kernels an entry point launches, without a GPU.

A process of its own loads the library behind a small recorder that stands in for the HIP runtime's launch
calls: a call runs its host checks and its choice of kernels, every launch is written down, and no kernel runs.
Pointers may be any aligned numbers; they are never followed."""
from __future__ import annotations

import json
import os
import re
import subprocess
import sys
import tempfile

import genomic_lm_amd as G

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

RECORDER = r"""
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
typedef struct { unsigned x, y, z; } dim3_t;
static struct known { const void* host; const char* name; } *known;      /* of every library of the process */
static int n_known, room;
static char text[1 << 16];
static dim3_t grid, block;
static size_t shared;
static void* stream;
const char* recorded(void) { return text; }
const char* name_of(int i) { return i < n_known ? known[i].name : 0; }
void forget(void) { text[0] = 0; }
void** __hipRegisterFatBinary(const void* data) { static void* h[1]; (void)data; return h; }
void __hipUnregisterFatBinary(void** m) { (void)m; }
void __hipRegisterFunction(void** m, const void* host, char* dev, const char* name, unsigned limit, void* a, void* b,
                           void* c, void* d, int* w) {
  (void)m; (void)dev; (void)limit; (void)a; (void)b; (void)c; (void)d; (void)w;
  if (n_known == room) known = realloc(known, (room = 2 * room + 1024) * sizeof *known);
  known[n_known].host = host;
  known[n_known++].name = name;
}
void __hipRegisterVar(void** m, void* v, char* h, char* d, int e, size_t s, int c, int g) {
  (void)m; (void)v; (void)h; (void)d; (void)e; (void)s; (void)c; (void)g;
}
int __hipPushCallConfiguration(dim3_t g, dim3_t b, size_t s, void* st) { grid = g; block = b; shared = s; stream = st; return 0; }
int __hipPopCallConfiguration(dim3_t* g, dim3_t* b, size_t* s, void** st) {
  *g = grid; *b = block; *s = shared; *st = stream;
  return 0;
}
int hipLaunchKernel(const void* f, dim3_t g, dim3_t b, void** args, size_t s, void* st) {
  const char* name = "?";
  (void)args; (void)s; (void)st;
  for (int i = 0; i < n_known; ++i)
    if (known[i].host == f) name = known[i].name;
  const size_t at = strlen(text);
  snprintf(text + at, sizeof text - at, "%s %u %u %u %u\n", name, g.x, g.y, g.z, b.x);
  return 0;
}
int hipGetLastError(void) { return 0; }
int hipGetDevice(int* d) { *d = 0; return 0; }
int hipGetSymbolAddress(void** p, const void* s) { (void)s; *p = 0; return 1; }
"""

CHILD = """
import ctypes, json, sys
recorder = ctypes.CDLL(sys.argv[1], ctypes.RTLD_GLOBAL)     # found before the library's own runtime
recorder.recorded.restype = recorder.name_of.restype = ctypes.c_char_p
import genomic_lm_amd as G
G.lib()
names, i = [], 0
while (name := recorder.name_of(i)) is not None:
    names.append(name.decode())
    i += 1
out = []
for name, args in json.load(sys.stdin):
    recorder.forget()
    status = getattr(G.lib(), name)(*args)
    out.append([status, recorder.recorded().decode().split("\\n")[:-1]])
json.dump([out, [n for n in names if n.startswith("_ZN5hyena")]], sys.stdout)
"""


def _kernel(name):
    """(kernel, template arguments) of a mangled name."""
    m = re.match(r"_ZN5hyenaL?(?:12_GLOBAL__N_1)?\d+([a-z_0-9]+?)(?:I(.*?)EEv|E)", name)
    assert m, name
    return m.group(1), tuple(int(v) for v in re.findall(r"L[ib](\d+)E", (m.group(2) or "") + "E"))


def _record(calls):
    with tempfile.TemporaryDirectory() as d:
        src, lib = os.path.join(d, "recorder.c"), os.path.join(d, "recorder.so")
        with open(src, "w") as f:
            f.write(RECORDER)
        subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", lib, src], check=True)
        r = subprocess.run([sys.executable, "-c", CHILD, lib], input=json.dumps(calls), capture_output=True, text=True,
                           cwd=ROOT, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return json.loads(r.stdout)


def launches(calls):
    """[(entry point, arguments)] -> [(status, [(kernel, template arguments, grid, threads)])]."""
    out = []
    for status, lines in _record(calls)[0]:
        found = []
        for line in lines:
            name, x, y, z, threads = line.split()
            found.append((*_kernel(name), (int(x), int(y), int(z)), int(threads)))
        out.append((status, found))
    return out


def library_kernels():
    """(kernel, template arguments) of every kernel of the library's namespace."""
    return [_kernel(name) for name in _record([])[1]]


FAR = 1 << 40                # an aligned place that is never followed
BF, F32, F8 = "bf16", "fp32", "e4m3"


def linear(T, K, N, out=BF, unaligned=False, group=128):
    runs = -(-K // 128)
    at = FAR + 1 if unaligned else FAR
    return ("hyena_linear_fp8", [at, K, FAR, runs if group else 1, group, FAR, FAR, None, FAR, N, T, N, K,
                                 G.BF16 if out == BF else G.F32, None])


def gated(T, K, I, out=BF, unaligned=False, weights=FAR):
    runs = -(-K // 128)
    at = FAR + 1 if unaligned else FAR
    head = [at, K, FAR, runs, 128, weights, weights, weights, weights, 1]
    if out == F8:
        need = G.gated_linear_fp8_workspace_size(T, I, K)
        return ("hyena_gated_linear_fp8_quant", head + [FAR, FAR, T, I, K, FAR if need else None, need, None])
    return ("hyena_gated_linear_fp8", head + [FAR, I, T, I, K, G.BF16 if out == BF else G.F32, None])
