"""Linear attention on the GPU where a loose bound would hide a fault: states that nothing is written to,
errors in the norm, gradients of log_a, calls from two threads."""
import ctypes
import subprocess

import pytest
import torch

import linattn_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU test"
    from gated_delta_rule_159_b200 import gdn2
    return gdn2


CALLER = r"""
#include <pthread.h>
#include <stddef.h>
#include <stdint.h>
typedef int (*fwd_t)(const void *, const void *, const void *, const void *, const float *, const int32_t *, void *,
                     float *, const void *, void *, size_t, void *);
struct call { fwd_t fn; const void *q, *k, *v, *la, *S0; void *o, *S, *ws, *stream; const void *dims; int64_t n, bad; };
static void *work(void *arg) {
  struct call *c = arg;
  for (int64_t i = 0; i < c->n; ++i)
    c->bad += c->fn(c->q, c->k, c->v, c->la, c->S0, NULL, c->o, c->S, c->dims, c->ws, 256, c->stream) != 0;
  return NULL;
}
void run(struct call *c, int threads) {
  pthread_t t[16];
  for (int i = 0; i < threads; ++i) pthread_create(&t[i], NULL, work, &c[i]);
  for (int i = 0; i < threads; ++i) pthread_join(t[i], NULL);
}
"""


class Call(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("fn", "q", "k", "v", "log_a", "S0", "o", "S", "ws", "stream", "dims")] + [
        ("n", ctypes.c_int64), ("bad", ctypes.c_int64)]


def test_threads_with_heads_of_two_sizes(g, tmp_path):
    """The fp32 run's shared memory differs by head size; no thread's launches may see another's."""
    src, so = tmp_path / "caller.c", tmp_path / "caller.so"
    src.write_text(CALLER)
    subprocess.check_call(["gcc", "-O2", "-shared", "-fPIC", "-pthread", str(src), "-o", str(so)])
    calls, kept = (Call * 4)(), []
    for i, d in enumerate((40, 128, 40, 128)):
        p = ref.problem((3,), 1, 1, d, d, F32, "token", True, seed=50 + d)[0]
        want = g.linattn_fwd(p["q"], p["k"], p["v"], p["log_a"], p["S0"])
        dims = g.LinattnDims(1, 3, 1, 1, d, d, g.F32, g.F32, 0, 0)
        o, S, ws = torch.empty_like(p["v"]), torch.empty_like(p["S0"]), torch.empty(256, dtype=torch.uint8, device="cuda")
        stream = torch.cuda.Stream()
        calls[i] = Call(ctypes.cast(g.lib.gdn2_linattn_fwd, ctypes.c_void_p).value,
                        *(p[x].data_ptr() for x in ("q", "k", "v", "log_a", "S0")), o.data_ptr(), S.data_ptr(), ws.data_ptr(),
                        stream.cuda_stream, ctypes.addressof(dims), 20000, 0)
        kept.append((p, want, o, S, ws, stream, dims))
    torch.cuda.synchronize()
    ctypes.CDLL(str(so)).run(calls, 4)
    torch.cuda.synchronize()
    for call, (_, want, o, S, *_) in zip(calls, kept):
        assert call.bad == 0
        assert torch.equal(o, want[0]) and torch.equal(S, want[1])
