"""A stand-in for the CUDA runtime, for tests of the host side without a GPU:
a small library that takes the place of the four calls a launch goes through,
so that no kernel runs and what a call would have launched can be looked at.

``run(body)`` runs Python code in a process of its own, with ``lib`` (the
library), ``launches`` (list of (shared bytes, limit, status, first ``arg_bytes``
bytes of the kernel's second argument)) and ``on_set_limit`` (a list: its function, if
any, runs once inside the next call that sets a kernel's shared-memory limit)
in its namespace, and returns what it printed.
"""
import os
import subprocess
import sys
import textwrap

SHIM = r"""
#include <stddef.h>
#include <string.h>
typedef struct { unsigned g[3], b[3]; size_t smem; } config;
static const void *fn[64];
static int limit[64], n_fn;
static void (*hook)(void);
static int (*seen)(size_t, int, int, void **);
void shim_hook(void (*h)(void)) { hook = h; }
void shim_seen(int (*s)(size_t, int, int, void **)) { seen = s; }
static int *of(const void *f) {
    for (int i = 0; i < n_fn; ++i) if (fn[i] == f) return &limit[i];
    fn[n_fn] = f; limit[n_fn] = 48 * 1024; return &limit[n_fn++];
}
int cudaGetDevice(int *d) { *d = 0; return 0; }
int cudaDeviceGetAttribute(int *v, int a, int d) { *v = 148; return 0; }
int cudaFuncSetAttribute(const void *f, int a, int v) {
    *of(f) = v;
    if (hook) { void (*h)(void) = hook; hook = 0; h(); }
    return 0;
}
int cudaLaunchKernelExC(const config *c, const void *f, void **args) {
    int status = c->smem > (size_t)*of(f) ? 1 : 0;
    if (seen) seen(c->smem, *of(f), status, args);
    return status;
}
"""

PRELUDE = r"""
import ctypes, sys
shim = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)  # found before the real runtime
lib = ctypes.CDLL(sys.argv[2])
launches, on_set_limit = [], []
arg_bytes = 0
P, I64, I, F64, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_double, ctypes.c_size_t
HOOK, SEEN = ctypes.CFUNCTYPE(None), ctypes.CFUNCTYPE(I, SZ, I, I, ctypes.POINTER(P))
@SEEN
def seen(smem, limit, status, args):
    launches.append((smem, limit, status, ctypes.string_at(args[1], arg_bytes) if arg_bytes else b""))
    return 0
@HOOK
def hook():
    if on_set_limit:
        on_set_limit.pop()()
shim.shim_seen(seen)
shim.shim_hook(hook)
DS_OK = 560
lib.ds_paged_plan.argtypes = [P, P, I, P, I64, I, I64, P, I, P, P, P, P, P, I64, P, P, SZ, P]
lib.ds_rope_append.argtypes = [P, I64, I, I64, I64, P, I, P, I, I, I, I, F64, I, P, I64, I, P, P, I, I64, P, P, SZ, P]
def rope(rows, nq, nkv, hd, rot, base, dtype=0):
    # addresses that nothing reads, far apart
    w = (nq + 2 * nkv) * hd
    at = [0x100000000 * (i + 1) for i in range(7)]
    return lib.ds_rope_append(at[0], rows * w, dtype, w, rows, at[1], 1, None, nq, nkv, hd, rot, base, 0, at[2],
                              rows * nq * hd, dtype, at[3], at[4], dtype, rows, at[5], at[6], 256, None)
"""


def run(body, tmp_path):
    from autoregressive_decode_step_gb300 import build
    lib = build.build()
    src, shim = os.path.join(tmp_path, "shim.c"), os.path.join(tmp_path, "libshim.so")
    with open(src, "w") as f:
        f.write(SHIM)
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", shim, src], check=True)
    r = subprocess.run([sys.executable, "-c", PRELUDE + textwrap.dedent(body), shim, lib], capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout
