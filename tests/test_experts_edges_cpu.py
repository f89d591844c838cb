"""CPU checks of calls at the edges of what is documented for the operators that
carry rows to experts and back and for the products with 4-bit weights: empty
batches, which packed rows are read, weights in strange places."""

import os
import re
import subprocess

import pytest

torch = pytest.importorskip("torch")

from trellis_quantized_moe_amd import exl3  # noqa: E402
from trellis_quantized_moe_amd.csrc import build as B  # noqa: E402


@pytest.mark.parametrize("topk", [1, 8])
def test_an_empty_batch_with_the_buffers_of_route_pack(monkeypatch, topk):
    """No rows, on the way that a program takes: alloc_meta's buffers hold at
    least one element each."""
    monkeypatch.setattr(exl3, "_stream", lambda: None)
    meta = exl3.alloc_meta(0, topk, 4, "cpu")
    assert meta["pos_of_pair"].numel() == 1
    meta = exl3.exl3_route_pack(torch.zeros(0, topk, dtype=torch.int32), torch.zeros(0, topk), 4,
                                meta)
    e = torch.zeros(0, 16)
    xs = exl3.exl3_permute(e, meta, topk)
    assert xs.shape == (0, 16)
    assert exl3.exl3_unpermute(xs, meta, topk, torch.zeros(0, topk)).shape == (0, 16)
    dy, dw = exl3.exl3_unpermute_backward(e, meta, topk, xs, torch.zeros(0, topk))
    assert dy.shape == (0, 16) and dw.shape == (0, topk)
    for t in (torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)):
        with pytest.raises(exl3.Exl3Error, match="pos_of_pair"):
            exl3.exl3_permute(e, {"pos_of_pair": t}, topk)


# ------------------------------------------------- which packed rows are read
HOST = r"""
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <math.h>
#include <sys/mman.h>
#include <algorithm>
#define __device__
#define __global__
#define __forceinline__ inline
#define __launch_bounds__(n)
using std::max;
using std::min;
struct Dim { unsigned x, y; };
static Dim threadIdx, blockIdx, blockDim, gridDim;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
static float bf16_bits_to_f32(uint16_t b) {
  return __builtin_bit_cast(float, (uint32_t)b << 16);
}
static float f16_bits_to_f32(uint16_t) { abort(); }  // no fp16 here
static uint32_t f32x2_to_out16(float, float, int) { abort(); }
@PARAMS@
@KERNEL@
// A row of y is a page. Those that no choice names can not be read.
template <int B>
static void check(int rows, int topk, unsigned seed, int dropped) {
  const int F = 1024, pairs = rows * topk;
  float *y = (float *)mmap(0, (size_t)pairs * 4096, PROT_READ | PROT_WRITE,
                           MAP_PRIVATE | MAP_ANONYMOUS, -1, 0);
  int32_t *pos = new int32_t[pairs];
  float *w = new float[pairs], *out = new float[rows * F];
  srand(seed);
  for (int i = 0; i < pairs; ++i) {
    pos[i] = i;
    w[i] = (float)(rand() % 9 - 4);
    for (int h = 0; h < F; ++h) y[i * F + h] = (float)(rand() % 17 - 8);
  }
  for (int i = pairs - 1; i > 0; --i) std::swap(pos[i], pos[rand() % (i + 1)]);
  const int32_t none[] = {-1, pairs, INT32_MAX, INT32_MIN};
  for (int i = 0; i < pairs; ++i)
    if (rand() % 100 < dropped || pos[i] == 0) {
      mprotect(y + pos[i] * F, 4096, PROT_NONE);
      pos[i] = none[rand() % 4];
    }
  MoveParams p{};
  p.pos = pos;
  p.rows = rows;
  p.topk = topk;
  p.pairs = pairs;
  p.features = F;
  p.x = y;
  p.ldx = F;
  p.w = w;
  p.w_dtype = 3;
  p.out = out;
  p.ldout = F;
  blockDim = {128, 2};
  gridDim = {1, 1};
  for (threadIdx.y = 0; threadIdx.y < 2; ++threadIdx.y)
    for (threadIdx.x = 0; threadIdx.x < 128; ++threadIdx.x) unpermute_kernel<3, 3, B, false>(p);
  for (int t = 0; t < rows; ++t)
    for (int h = 0; h < F; ++h) {
      float s = 0;
      for (int j = 0; j < topk; ++j) {
        const int q = pos[t * topk + j];
        if (q >= 0 && q < pairs) s += w[t * topk + j] * y[q * F + h];
      }
      if (s != out[t * F + h]) exit(printf("row %d\n", t));
    }
  munmap(y, (size_t)pairs * 4096);
}
int main() {
  for (int dropped : {0, 30, 100})
    for (unsigned seed = 0; seed < 3; ++seed) {
      check<1>(3, 1, seed, dropped);
      check<2>(5, 2, seed, dropped);
      check<4>(3, 3, seed, dropped);
      check<8>(3, 8, seed, dropped);
      check<8>(4, 13, seed, dropped);
      check<8>(2, 17, seed, dropped);
    }
  printf("all read\n");
}
"""


def test_unpermute_reads_the_rows_of_choices_alone(tmp_path):
    """The kernel's source, built for the host, over packed rows of a page each:
    a read of one that no choice names ends the program."""
    clang = os.path.join(os.path.dirname(os.path.realpath(B.HIPCC)), "..", "lib", "llvm", "bin",
                         "clang++")
    if not os.path.exists(clang):
        pytest.skip("no clang++")
    with open(os.path.join(B.HERE, "permute.hip")) as f:
        src = f.read()
    with open(os.path.join(B.HERE, "kernels.hpp")) as f:
        params = re.search(r"^struct MoveParams \{.*?^\};", f.read(), re.S | re.M).group(0)
    kernel = src[src.index("constexpr int kThreads"):src.index("// DY: type of y and dy")]
    assert "unpermute_kernel" in kernel
    cpp, exe = tmp_path / "host.cpp", tmp_path / "host"
    cpp.write_text(HOST.replace("@PARAMS@", params).replace("@KERNEL@", kernel))
    r = subprocess.run([clang, "-O1", "-std=c++17", "-fwrapv", str(cpp), "-o", str(exe)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "all read\n", (r.returncode, r.stdout)


# ------------------------------------------------------- weights laid out
def test_experts_an_odd_number_of_bytes_apart():
    """Every expert's weights are read as words, wherever they start; also where
    a step of the layout holds one expert."""
    g = torch.Generator().manual_seed(1)
    E, N, K = 2, 2056, 32768  # a step holds at most 2^27 weights: one expert
    q = torch.randint(0, 256, (E, N * K // 2), generator=g, dtype=torch.uint8)
    s = torch.rand(E, N, K // 128, generator=g).half()
    want = exl3.DeviceW4(q.view(E, N, K // 2), s).q
    for first, more in ((0, 1), (0, 2), (1, 3), (2, 5)):
        far = torch.zeros(first + E * (N * K // 2 + more), dtype=torch.uint8)
        apart = far[first:].view(E, -1)[:, :N * K // 2]
        apart.copy_(q)
        got = exl3.DeviceW4(apart.view(E, N, K // 2), s).q
        assert torch.equal(got, want), (first, more)


@pytest.mark.parametrize("E,N,K", [(1, 4, 64), (2, 12, 64), (1, 65544, 32), (1, 8, 65568),
                                   (1025, 8, 32), ((1 << 32) + 1, 8, 32)])
def test_weights_that_no_product_takes_are_refused_at_once(E, N, K):
    """Outputs that are no multiple of 8 and sizes past the limits: at the
    layout, not at the first product."""
    q = torch.zeros(1, 1, K // 2, dtype=torch.uint8).expand(E, N, K // 2)
    s = torch.ones(1, 1, 1).half().expand(E, N, K // 32)
    with pytest.raises(exl3.Exl3Error, match="status -[37]|out of range"):
        exl3.DeviceW4(q, s)
