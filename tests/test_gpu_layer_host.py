"""Host side of the launches: calls from two host threads at once, and a call after one
whose launch was refused."""
import ctypes
import os
import subprocess

import pytest
import torch

import linear_attention_lm_b200 as lab
from linear_attention_lm_b200 import build as lab_build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lab_build.build()
    lab.load_library()
    torch.cuda.set_device(0)


def normal(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


HAMMER = r"""
#include <atomic>
#include <thread>
#include "based.h"
struct Call { int kind; void* p[12]; long long n[8]; void* stream; };
static int one(const Call& c) {
  void* const* p = c.p; const long long* n = c.n;
  typedef float F;
  const based_dtype_t dt = BASED_F32;
  if (c.kind == 0)
    return based_layernorm_bwd(p[0], p[1], (F*)p[2], (F*)p[3], (F*)p[4], 0, (F*)p[5], (F*)p[6], (F*)p[7],
                               n[0], n[1], dt, p[8], n[2], c.stream);
  if (c.kind == 1)
    return based_gatedrec_bwd(p[0], p[1], p[2], (F*)p[3], 0, (F*)p[4], (F*)p[5], (F*)p[6], 0, n[0], n[1],
                              n[2], dt, c.stream);
  if (c.kind == 2)
    return based_window_attn_fwd(p[0], p[1], p[2], p[3], n[0], n[1], n[2], n[3], 64, dt, c.stream);
  return based_decode_step(0, 0, 0, 0, 0, 0, p[0], p[1], p[2], p[3], p[4], p[5], 67, n[0], 0, 16, 64, n[1],
                           n[2], 64, dt, 1e-6f, c.stream);
}
// Two threads repeat a call each, at once; the number of calls that were not accepted.
extern "C" int hammer(const Call* calls, int times) {
  std::atomic<int> refused(0), ready(0);
  auto work = [&](const Call& c) {
    ++ready;
    while (ready < 2) {}
    for (int i = 0; i < times; ++i) refused += one(c) != BASED_OK;
  };
  std::thread other(work, calls[1]);
  work(calls[0]);
  other.join();
  return refused;
}
"""


class Call(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("p", ctypes.c_void_p * 12), ("n", ctypes.c_longlong * 8),
                ("stream", ctypes.c_void_p)]


@pytest.fixture(scope="module")
def hammer(tmp_path_factory):
    d = tmp_path_factory.mktemp("hammer")
    (d / "hammer.cpp").write_text(HAMMER)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-pthread", "-I", lab_build.INCLUDE,
                    "-o", str(d / "hammer.so"), str(d / "hammer.cpp"), lab.LIB_PATH,
                    "-Wl,-rpath," + os.path.dirname(lab.LIB_PATH)], check=True)
    return ctypes.CDLL(str(d / "hammer.so")).hammer


def layernorm_gradient(D):
    """Width D decides the kernel's shared memory (about 50 KB at 517, 96 KB at 999)."""
    x, dy, w = normal(1, 40, D), normal(2, 40, D), normal(3, D)
    _, mean, rstd = lab.layernorm(x, w, return_stats=True)
    outs = [torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)]
    size = lab.based_layernorm_bwd_workspace_bytes(40, D)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    return 0, [dy, x, w, mean, rstd, *outs, ws], [40, D, size], outs


def recurrence_gradient(L):
    x, g, dy = (normal(i, 64, L, 320) for i in (4, 5, 6))
    _, chunks = lab.gatedrec(x, g, for_grad=True)
    outs = [torch.empty_like(x), torch.empty_like(x), torch.empty(64, 320, device="cuda")]
    return 1, [x, g, dy, chunks, *outs], [64, L, 320], outs


def window(d_head):
    q, k, v = (normal(i, 1, 2, 40, d_head) for i in (7, 8, 9))
    out = torch.empty_like(q)
    return 2, [q, k, v, out], [1, 2, 40, d_head], [out]


def decode(d_head):
    wq, wk, wv = (normal(i, 2, 2, d_head) for i in (10, 11, 12))
    rings = [normal(13 + i, 2, 2, 64, d_head) for i in range(2)]
    out = torch.empty_like(wq)
    return 3, [wq, wk, wv, *rings, out], [2, 2, d_head], [out]


@pytest.mark.parametrize("make,sizes", [(layernorm_gradient, (517, 999)), (recurrence_gradient, (8, 47)),
                                        (window, (64, 128)), (decode, (64, 128))])
def test_two_host_threads(hammer, make, sizes):
    """Each thread repeats its own size on its own stream: no call is refused, and the
    bits are those of a call alone."""
    made = [make(s) for s in sizes]
    streams = [torch.cuda.Stream() for _ in made]
    calls = (Call * 2)(*[Call(kind, (ctypes.c_void_p * 12)(*[t.data_ptr() for t in ts]),
                              (ctypes.c_longlong * 8)(*n), st.cuda_stream)
                         for (kind, ts, n, _), st in zip(made, streams)])
    torch.cuda.synchronize()
    want = []
    for c, (_, _, _, outs) in zip(calls, made):
        assert hammer((Call * 2)(c, c), 1) == 0  # the same call twice: nothing to disagree about
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    refused = hammer(calls, 20000)
    torch.cuda.synchronize()
    assert refused == 0
    for (_, _, _, outs), w in zip(made, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, w))
    assert lab.based_get_device_error() == 0


def test_a_refused_launch_leaves_the_next_call_alone():
    """A launch on the legacy stream is refused by the runtime while another stream, which
    that one waits for, is being captured; the calls after it say nothing of it."""
    rt = ctypes.CDLL("libcudart.so.12")
    x, g, h = (normal(i, 4, 64) for i in range(3))
    y = torch.empty_like(x)
    held = h.clone()
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    torch.cuda.synchronize()
    assert rt.cudaStreamCreate(ctypes.byref(stream)) == 0
    assert rt.cudaStreamBeginCapture(stream, 1) == 0
    try:
        with pytest.raises(lab.BasedError) as e:
            lab.based_gatedrec_step(x, g, h, y, stream=0)
    finally:
        rt.cudaStreamEndCapture(stream, ctypes.byref(graph))
        rt.cudaStreamDestroy(stream)
        rt.cudaGetLastError()
    assert e.value.status == 3
    lab.based_gatedrec_step(x, g, h, y)
    torch.cuda.synchronize()
    want = held * torch.sigmoid(g) + x * torch.sigmoid(-g)
    assert torch.allclose(h, want, rtol=1e-5, atol=1e-5)
