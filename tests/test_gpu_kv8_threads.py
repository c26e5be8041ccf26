"""Block selection called from two host threads at once (needs a B200).

The kernel's shared memory grows with the row, and the library asks the
runtime for it once. Two threads that meet there with rows of different
lengths must both be served, and so must every call after them. A process of
its own, where nothing has been asked for yet; the threads are started in C,
behind a spinning barrier, so that they do meet.
"""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

MEET = r"""
#include <pthread.h>
#include <stdatomic.h>
typedef int (*call_t)(const void*, const void*, const void*, const void*,
                      const void*, const void*, const void*, int, int, int,
                      int, int, int, int, int, int, int, int, void*, void*,
                      void*);
typedef struct {
  call_t call;
  const void *q, *kb, *ks, *start, *len, *pos, *table;
  void *blocks, *scores;
  int G, L, status;
  atomic_int* here;
} one_t;
static void* run(void* p) {
  one_t* x = (one_t*)p;
  atomic_fetch_add(x->here, 1);
  while (atomic_load(x->here) < 2) {}
  x->status = x->call(x->q, x->kb, x->ks, x->start, x->len, x->pos, x->table,
                      4, 1, x->L, x->G, 1, 128, 0, 0, 2, 1, 1, x->blocks,
                      x->scores, 0);
  return 0;
}
/* 100 * status of the shorter row's call + status of the longer one's */
int meet(void* call, void** t, int G, int short_len, int long_len) {
  atomic_int here = 0;
  one_t x[2];
  pthread_t th[2];
  for (int i = 0; i < 2; ++i) {
    one_t y = {(call_t)call, t[0], t[1], t[2], t[3], t[4], t[5], t[6],
               t[7 + 2 * i], t[8 + 2 * i], G, i ? long_len : short_len, -1,
               &here};
    x[i] = y;
    if (pthread_create(&th[i], 0, run, &x[i])) return -1;
  }
  for (int i = 0; i < 2; ++i) pthread_join(th[i], 0);
  return 100 * x[0].status + x[1].status;
}
"""

CHILD = r"""
import ctypes, sys
import torch
from long_context_blockwise_causal_b200 import ops
meet = ctypes.CDLL(sys.argv[1]).meet
meet.argtypes = [ctypes.c_void_p, ctypes.c_void_p] + [ctypes.c_int] * 3
L = ops.lib()
call = ctypes.cast(L.lwm_kv8_select, ctypes.c_void_p)
n = 32768                                     # blocks of the longest row
kb = torch.randint(-127, 128, (n, 2, 128), dtype=torch.int8, device="cuda")
ks = torch.rand(n, device="cuda")
q = torch.randn(16, 128, device="cuda").bfloat16()
i32 = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")
start, length, pos = i32(0), i32(n * 128), i32(1)
table = ops.rope_table(1e4, 4)
outs = [torch.empty(2, dtype=torch.int32, device="cuda") for _ in range(4)]
ptrs = (ctypes.c_void_p * 11)(*(t.data_ptr() for t in (
    q, kb, ks, start, length, pos, table, *outs)))
torch.cuda.synchronize()
bad = []
for G in (1, 2, 3, 7, 16):
    for at in range(12000, n - 200, 200):
        s = meet(call, ptrs, G, at * 128, (at + 150) * 128)
        # and a call after them, as long as the longer one
        t = L.lwm_kv8_select(
            q.data_ptr(), kb.data_ptr(), ks.data_ptr(), start.data_ptr(),
            length.data_ptr(), pos.data_ptr(), table.data_ptr(), 4, 1,
            (at + 150) * 128, G, 1, 128, 0, 0, 2, 1, 1, outs[0].data_ptr(),
            outs[1].data_ptr(), 0)
        if s or t:
            bad.append((G, at, s, t))
torch.cuda.synchronize()
print("refused", len(bad), bad[:4])
sys.exit(1 if bad else 0)
"""


def test_rows_of_two_lengths_from_two_threads(cuda_dev, tmp_path):
    src, lib = tmp_path / "meet.c", tmp_path / "meet.so"
    src.write_text(MEET)
    subprocess.run(["gcc", "-O2", "-shared", "-fPIC", "-pthread", str(src),
                    "-o", str(lib)], check=True)
    r = subprocess.run([sys.executable, "-c", CHILD, str(lib)], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
