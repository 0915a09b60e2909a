"""Several host threads in the same calls at once, with sizes that need
different amounts of shared memory: no call is refused, each gets the result
that it gets alone.  The threads are the C ABI's own users, without the
interpreter's lock between them: a small program compiled here."""
import ctypes
import os
import shutil
import subprocess
import threading
import time

import pytest
import torch

from _parity import dev

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROUNDS = 3000

SOURCE = r"""
#include <atomic>
#include <thread>
#include <vector>
#include "include/moe_gb300.h"

// What one thread calls again and again.
struct Job {
  int kind, T, k, E, n, K, N, R, dtype;
  const void *x, *a, *b, *base, *ids;
  void *out, *out2, *out3, *out4, *ws;
  size_t ws_bytes;
  void* stream;
};

extern "C" int call(const Job* j, decltype(&moe_router_logits) logits,
                    decltype(&moe_permute_masked) permute, decltype(&moe_lora_apply) lora) {
  auto u16 = [](const void* p) { return static_cast<const uint16_t*>(p); };
  auto i32 = [](const void* p) { return static_cast<const int32_t*>(p); };
  auto o32 = [](void* p) { return static_cast<int32_t*>(p); };
  if (j->kind == 0)
    return logits(u16(j->x), static_cast<const float*>(j->a), nullptr, 1.0f, j->T, j->K, j->E,
                  static_cast<float*>(j->out), j->stream);
  if (j->kind == 1)
    return permute(i32(j->ids), i32(j->x), j->T, j->k, j->E, -1, o32(j->out), o32(j->out2),
                   o32(j->out3), o32(j->out4), j->stream);
  return lora(u16(j->x), 1, i32(j->ids), nullptr, nullptr, nullptr, j->T, 1, 1, j->n, j->K, j->N,
              j->R, u16(j->a), u16(j->b), nullptr, j->base, j->dtype, MOE_EPILOGUE_RAW, j->dtype,
              j->out, j->ws, j->ws_bytes, j->stream);
}

// Every job in a thread of its own: how many calls were refused.
extern "C" int together(const Job* jobs, int n, int rounds, decltype(&moe_router_logits) logits,
                        decltype(&moe_permute_masked) permute, decltype(&moe_lora_apply) lora) {
  std::atomic<int> waiting(n), refused(0);
  std::vector<std::thread> threads;
  for (int i = 0; i < n; ++i)
    threads.emplace_back([&, i] {
      --waiting;
      while (waiting.load() > 0) std::this_thread::yield();
      for (int r = 0; r < rounds; ++r) refused += call(jobs + i, logits, permute, lora) != 0;
    });
  for (auto& t : threads) t.join();
  return refused.load();
}
"""

POINTERS = ["x", "a", "b", "base", "ids", "out", "out2", "out3", "out4", "ws"]


class Job(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in ("kind", "T", "k", "E", "n", "K", "N", "R", "dtype")]
                + [(n, ctypes.c_void_p) for n in POINTERS]
                + [("ws_bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p)])


@pytest.fixture(scope="module")
def hammer(tmp_path_factory, cuda_lib):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("threads")
    (d / "threads.cpp").write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-pthread", "-I", ROOT,
                    str(d / "threads.cpp"), "-o", str(d / "threads.so")], check=True)
    so = ctypes.CDLL(str(d / "threads.so"))
    fns = [ctypes.cast(getattr(cuda_lib.lib(), n), ctypes.c_void_p)
           for n in ("moe_router_logits", "moe_permute_masked", "moe_lora_apply")]

    def together(jobs):
        """jobs: (fields of Job, the tensors of its pointers, its results)."""
        streams = [torch.cuda.Stream() for _ in jobs]
        arr = (Job * len(jobs))()
        for j, (fields, tensors, _), s in zip(arr, jobs, streams):
            for name, v in fields.items():
                setattr(j, name, v)
            for name, t in tensors.items():
                setattr(j, name, t.data_ptr())
            j.stream = s.cuda_stream
        want = []
        for j, (_, _, results) in zip(arr, jobs):
            assert so.call(ctypes.byref(j), *fns) == 0
            torch.cuda.synchronize()
            want.append([t.clone() for t in results])
            for t in results:
                t.zero_()
        torch.cuda.synchronize()
        assert so.together(arr, len(jobs), ROUNDS, *fns) == 0
        torch.cuda.synchronize()
        for (_, _, results), ref in zip(jobs, want):
            assert all(torch.equal(a, b) for a, b in zip(results, ref))
    return together


def test_router_logits_of_several_widths(hammer):
    def job(E, T=4, K=64):
        x = torch.randn((T, K), device=dev()).bfloat16()
        w = torch.randn((E, K), device=dev())
        out = torch.empty((T, E), device=dev())
        return dict(kind=0, T=T, K=K, E=E), dict(x=x, a=w, out=out), [out]
    hammer([job(1024), job(800), job(1000), job(64)])


def test_grouping_of_several_widths(hammer):
    def job(E, T=16, k=4):
        ids = torch.randint(-1, E, (T, k), dtype=torch.int32, device=dev())
        kd = torch.full((1,), k, dtype=torch.int32, device=dev())
        outs = [torch.zeros(m, dtype=torch.int32, device=dev()) for m in (E, E + 1, T * k, T * k)]
        names = dict(zip(("out", "out2", "out3", "out4"), outs))
        return dict(kind=1, T=T, k=k, E=E), dict(x=kd, ids=ids, **names), outs
    hammer([job(1024), job(400), job(700), job(8)])


def test_grouped_adapters_of_several_counts_and_ranks(hammer, cuda_lib):
    def job(n, R, dtype, T=1024, K=256, N=128):
        g = torch.Generator(device=dev())
        g.manual_seed(n)
        x = torch.randn((T, K), generator=g, device=dev()).bfloat16()
        a = (torch.randn((n, R, K), generator=g, device=dev()) * K ** -0.5).bfloat16()
        b = torch.randn((n, N, R), generator=g, device=dev()).bfloat16()
        base = torch.randn((T, N), generator=g, device=dev()).to(dtype)
        ids = torch.randint(-1, n, (T,), generator=g, device=dev(), dtype=torch.int32)
        size = cuda_lib.moe_lora_workspace_size(T, 1, 1, n, R)
        ws = torch.empty(size, dtype=torch.uint8, device=dev())
        out = torch.empty_like(base)
        dt = cuda_lib.DTYPE_BF16 if dtype == torch.bfloat16 else cuda_lib.DTYPE_F32
        return (dict(kind=2, T=T, n=n, K=K, N=N, R=R, dtype=dt, ws_bytes=size),
                dict(x=x, a=a, b=b, base=base, ids=ids, out=out, ws=ws), [out])
    hammer([job(2000, 32, torch.float32), job(700, 32, torch.float32),
             job(40, 72, torch.float32), job(1200, 128, torch.float32),
             job(30, 128, torch.bfloat16), job(31, 72, torch.bfloat16)])


def test_a_call_that_waits_for_its_queue_leaves_the_interpreter_free(cuda_lib):
    """A stream is kept busy for some half a second while one thread fills its
    queue; this thread goes on meanwhile."""
    l = torch.randn((8, 64), device=dev())
    outs = [t.clone() for t in cuda_lib.moe_route_scored(l, 4)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    spent = []

    def fill():
        with torch.cuda.stream(side):
            torch.cuda._sleep(1_000_000_000)
            t0 = time.perf_counter()
            for _ in range(6000):  # several times what a queue takes
                cuda_lib.moe_route_scored(l, 4, topk_ids=outs[0], topk_w=outs[1], k_dev=outs[2])
            spent.append(time.perf_counter() - t0)

    worker = threading.Thread(target=fill)
    longest, last = 0.0, time.perf_counter()
    worker.start()
    while worker.is_alive():
        time.sleep(0.001)
        now = time.perf_counter()
        longest, last = max(longest, now - last), now
    worker.join()
    torch.cuda.synchronize()
    assert spent[0] > 0.2      # the queue was full and the thread waited
    assert longest < spent[0] / 2
