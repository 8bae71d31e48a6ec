"""What nwc_attend asks of the runtime when several threads call it (no GPU): a
shim in the runtime's place records and answers."""
import os
import subprocess
import sys

import decode_gemv_byte_amd as nwc

# A runtime that enforces the LDS allowance of a kernel as it stands at the
# launch, and that lets another caller in between allowance and launch.
SHIM = r"""
#include <stddef.h>
typedef struct { unsigned x, y, z; } dim3;
static struct { const void* f; int most; } allowed[64];
int sets, launches;
void (*between)(void);
static int* of(const void* f) {
  int i = 0;
  while (allowed[i].f && allowed[i].f != f) ++i;
  allowed[i].f = f;
  return &allowed[i].most;
}
int hipGetDevice(int* d) { *d = 0; return 0; }
int hipFuncSetAttribute(const void* f, int attr, int value) {
  (void)attr;
  ++sets;
  *of(f) = value;
  return 0;
}
int hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t lds, void* stream) {
  (void)grid; (void)block; (void)args; (void)stream;
  void (*call)(void) = between;
  between = NULL;
  if (call) call();
  ++launches;
  return lds > 65536 && lds > (size_t)*of(f);
}
"""

SCRIPT = r"""
import ctypes, sys
shim, lib = ctypes.CDLL(sys.argv[1]), ctypes.CDLL(sys.argv[2])
u16, u32, u64, p = ctypes.c_uint16, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_void_p
class Cache(ctypes.Structure):
    _fields_ = [("k", p), ("v", p), ("n_pages", u64), ("page_stride", u64), ("kv_heads", u32), ("head_dim", u32),
                ("page_len", u32), ("reserved", u32)]
class Table(ctypes.Structure):
    _fields_ = [("ids", p), ("ld", u64), ("rows", u32), ("cols", u32)]
A = 0x100000                                  # addresses that nothing reads
def attend(rows, cols, d=128):
    c, t = Cache(A, A, 4, 8 * 64 * d, 8, d, 64, 0), Table(A, cols, rows, cols)
    return lib.nwc_attend(ctypes.byref(c), ctypes.byref(t), None, p(A), p(A), u64(32 * d), u32(32), ctypes.c_float(0.1),
                          p(2 * A), u64(32 * d), p(A), ctypes.c_size_t(1 << 40), None)
inner = []
back = ctypes.CFUNCTYPE(None)(lambda: inner.append(attend(1, 4096)))
ctypes.c_void_p.in_dll(shim, "between").value = ctypes.cast(back, p).value
outer = attend(4096, 4096)                    # a larger plan in LDS than the call in between has
sets = ctypes.c_int.in_dll(shim, "sets").value
again = [attend(rows, 4096) for rows in (4096, 1, 700)]
print(outer, inner, again, ctypes.c_int.in_dll(shim, "sets").value - sets, ctypes.c_int.in_dll(shim, "launches").value)
"""


def test_a_smaller_call_between_allowance_and_launch(tmp_path):
    src, so = tmp_path / "shim.c", tmp_path / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", str(so), str(src)], check=True)
    env = dict(os.environ, LD_PRELOAD=":".join([str(so)] + [x for x in [os.environ.get("LD_PRELOAD")] if x]))
    r = subprocess.run([sys.executable, "-c", SCRIPT, str(so), nwc.LIB_PATH], env=env, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    # every call got its LDS, and calls after the first ask for nothing
    assert r.stdout.strip() == "0 [0] [0, 0, 0] 0 10"
