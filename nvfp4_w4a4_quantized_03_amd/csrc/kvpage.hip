// The paged KV cache of a serving step, for gfx950: block tables, positions
// and slots built on the device from request lengths, and the write of new
// keys and values into their slots.
//
// Tables.  With c_r tokens cached and n_r new ones, request r holds
// ceil(c_r / P) pages and needs need_r = max(0, min(ceil((c_r + n_r) / P), W)
// - ceil(c_r / P)) more, taken from the free list in request order, so its
// first one is entry sum_{s < r} need_s.  Token t of the step belongs to the
// last r with cu_r <= t (cu the exclusive prefix sums of n) and stands at
// position c_r + t - cu_r.  Everything follows from two prefix sums over the
// requests, which every workgroup computes for itself in blocks of 256 (two
// loads a request and a scan: cheaper than a second launch or a grid-wide
// wait); a page's table entry is written by the thread of its first token,
// and a slot on a fresh page comes from the free list and not from the
// table, so no workgroup reads what another one writes.  Bound by latency:
// the loads of the lengths, the scan, and one dependent load of a page id
// (3.6 us for 32 decodes, 4.7 us for 256 requests of 32768 tokens together).
//
// Write.  One lane per 16 elements of a token's K or V row (16 or 32 bytes
// stored), consecutive lanes on consecutive elements: HBM-bound (32768 tokens
// of 4 heads of 256, bf16 to E4M3: 38 us, 5.3 TB/s; float32 to E4M3: 64 us,
// 5.2 TB/s; float32 to bf16: 81 us, 5.0 TB/s; bf16 to bf16: 57 us, 4.7 TB/s;
// 32 tokens: 3.8 us, a launch).  The FP8 form is the exact cast of fp8kv.hip.  Measured and not
// taken: cached stores (42 us), K and V of a group by one lane (40 us).
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "internal.h"
#include "kv_device.h"

namespace nvfp4 {
namespace {

constexpr int kTableThreads = 256;

// Inclusive scan of one value per thread over the workgroup; *total gets the
// sum.  `part` holds one word per wave and is free again after the call.
__device__ __forceinline__ int64_t scan256(int64_t v, int64_t* part, int64_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t o = __shfl_up(v, off);
    if (lane >= off) v += o;
  }
  if (lane == 63) part[wave] = v;
  __syncthreads();
  int64_t before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kTableThreads / 64; ++w) {
    const int64_t p = part[w];
    if (w < wave) before += p;
    sum += p;
  }
  *total = sum;
  __syncthreads();
  return v + before;
}

__global__ void __launch_bounds__(kTableThreads)
page_tables_kernel(const int32_t* __restrict__ new_lens, const int32_t* __restrict__ cached_lens,
                   int64_t n_requests, int32_t* __restrict__ table, int64_t cols, int64_t ld,
                   const int32_t* __restrict__ free_pages, int64_t n_free, FastDiv page,
                   int64_t n_tokens, int32_t* __restrict__ cu_new, int32_t* __restrict__ kv_lens,
                   int32_t* __restrict__ positions, int64_t* __restrict__ slots,
                   int32_t* __restrict__ pages_used) {
  __shared__ int64_t s_cu[kTableThreads + 1];      // first token of each request
  __shared__ int64_t s_first[kTableThreads];       // its first entry of the free list
  __shared__ int32_t s_cached[kTableThreads];
  __shared__ int64_t part[kTableThreads / 64];
  constexpr int64_t kMost = 0x7FFFFFFF;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kTableThreads + threadIdx.x;
  const unsigned psize = page.d;
  int64_t cu0 = 0, used0 = 0;                      // sums over the blocks before
  int32_t position = -1;
  int64_t slot = -1;
  for (int64_t b0 = 0; b0 < n_requests; b0 += kTableThreads) {
    const int64_t i = b0 + threadIdx.x;
    const bool real = i < n_requests;
    int64_t n = real ? new_lens[i] : 0, c = real ? cached_lens[i] : 0;
    n = n > 0 ? n : 0;
    c = c > 0 ? c : 0;
    n = n < kMost - c ? n : kMost - c;             // lengths stay below 2^31
    const unsigned kv = static_cast<unsigned>(c + n);
    // ceil(x / P) for x > 0 as floor((x - 1) / P) + 1
    const int64_t held = c ? page.div(static_cast<unsigned>(c) - 1u) + 1 : 0;
    const int64_t all = kv ? page.div(kv - 1u) + 1 : 0;
    const int64_t want = all < cols ? all : cols;
    const int64_t need = want > held ? want - held : 0;
    int64_t sum_n, sum_need;
    const int64_t cu = cu0 + scan256(n, part, &sum_n) - n;
    const int64_t first = used0 + scan256(need, part, &sum_need) - need;
    s_cu[threadIdx.x] = cu;
    s_first[threadIdx.x] = first;
    s_cached[threadIdx.x] = static_cast<int32_t>(c);
    if (threadIdx.x == 0) s_cu[kTableThreads] = cu0 + sum_n;
    // one workgroup writes each block's lengths and offsets
    if ((b0 / kTableThreads) % gridDim.x == blockIdx.x && real) {
      cu_new[i] = static_cast<int32_t>(cu < kMost ? cu : kMost);
      kv_lens[i] = static_cast<int32_t>(kv);
    }
    __syncthreads();
    if (t < n_tokens && t >= s_cu[0] && t < s_cu[kTableThreads]) {
      int lo = 0, hi = kTableThreads;              // s_cu[lo] <= t < s_cu[hi]
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= t) lo = mid; else hi = mid;
      }
      const int32_t cached = s_cached[lo];
      const unsigned pos = static_cast<unsigned>(cached + (t - s_cu[lo]));
      const int64_t blk = page.div(pos);
      const unsigned off = pos - static_cast<unsigned>(blk) * psize;
      const int64_t held_lo = cached ? page.div(static_cast<unsigned>(cached) - 1u) + 1 : 0;
      position = static_cast<int32_t>(pos);
      int64_t id = -1;
      if (blk < cols) {
        int32_t* entry = table + (b0 + lo) * ld + blk;
        if (blk < held_lo) {
          id = *entry;
        } else {
          const int64_t at = s_first[lo] + blk - held_lo;
          id = at < n_free ? free_pages[at] : -1;
          if (off == 0) *entry = static_cast<int32_t>(id);
        }
      }
      slot = id >= 0 ? id * psize + off : -1;
    }
    __syncthreads();
    cu0 += sum_n;
    used0 += sum_need;
  }
  if (t < n_tokens) {
    positions[t] = position;
    slots[t] = slot;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    cu_new[n_requests] = static_cast<int32_t>(cu0 < kMost ? cu0 : kMost);
    *pages_used = static_cast<int32_t>(used0 < kMost ? used0 : kMost);
  }
}

struct WriteArgs {
  const uint8_t* x[2];       // K and V
  uint8_t* cache[2];
  int64_t x_token[2], x_head[2];              // bytes
  int64_t page_stride, head_stride, token_stride;   // bytes
  const float* scale[2];
  const int64_t* slots;
  int64_t n_slots;           // n_pages * page_size
  unsigned groups;           // n_tokens * per_token
  FastDiv per_token, per_head, page;          // 16-element groups; tokens
};

template <int DTYPE, bool FP8>
__global__ void __launch_bounds__(256) page_write_kernel(WriteArgs a) {
  constexpr int64_t kBytes = 16 * (DTYPE == kDtypeF32 ? 4 : 2);
  const int which = blockIdx.y;
  const unsigned g = blockIdx.x * 256u + threadIdx.x;
  if (g >= a.groups) return;
  const unsigned t = a.per_token.div(g), in_token = g - t * a.per_token.d;
  const unsigned h = a.per_head.div(in_token), in_head = in_token - h * a.per_head.d;
  const int64_t slot = a.slots[t];
  if (slot < 0 || slot >= a.n_slots) return;
  const int64_t id = slot < 0x7FFFFFFF ? a.page.div(static_cast<unsigned>(slot))
                                       : slot / a.page.d;
  const int64_t off = slot - id * a.page.d;
  const uint8_t* src = a.x[which] + t * a.x_token[which] + h * a.x_head[which] + in_head * kBytes;
  uint8_t* dst = a.cache[which] + id * a.page_stride + h * a.head_stride + off * a.token_stride +
                 in_head * (FP8 ? 16 : 32);
  if constexpr (FP8) {
    const float s = *a.scale[which];
    const bool normal = s >= 0x1p-100f && s <= 0x1p100f;
    const float r = normal ? __builtin_amdgcn_rcpf(s) : 0.0f;    // within 2^-22 of 1 / s
    kv_cast_group<DTYPE>(src, dst, !(s > 0.0f), normal, r * (1.0f - 0x1p-18f),
                         r * (1.0f + 0x1p-18f), static_cast<double>(s));
  } else if constexpr (DTYPE == kDtypeF32) {
    float v[16];
    load16<DTYPE>(src, v);
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    unsigned w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const f32x2 p = {v[2 * i], v[2 * i + 1]};
      w[i] = __builtin_bit_cast(unsigned, __builtin_convertvector(p, bf16x2));   // RNE
    }
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
    const uint4 lo = reinterpret_cast<const uint4*>(src)[0];
    const uint4 hi = reinterpret_cast<const uint4*>(src)[1];
    reinterpret_cast<uint4*>(dst)[0] = lo;
    reinterpret_cast<uint4*>(dst)[1] = hi;
  }
}

}  // namespace

hipError_t launch_page_tables(const int32_t* new_lens, const int32_t* cached_lens,
                              int64_t n_requests, int32_t* block_table, int64_t cols, int64_t ld,
                              const int32_t* free_pages, int64_t n_free, int64_t page_size,
                              int64_t n_tokens, int32_t* cu_new, int32_t* kv_lens,
                              int32_t* positions, int64_t* slots, int32_t* pages_used,
                              hipStream_t stream) {
  const int64_t wgs = (n_tokens + kTableThreads - 1) / kTableThreads;
  page_tables_kernel<<<static_cast<unsigned>(wgs > 0 ? wgs : 1), kTableThreads, 0, stream>>>(
      new_lens, cached_lens, n_requests, block_table, cols, ld, free_pages, n_free,
      FastDiv::of(static_cast<unsigned>(page_size)), n_tokens, cu_new, kv_lens, positions, slots,
      pages_used);
  return hipGetLastError();
}

hipError_t launch_page_write(const KvRows& k, const KvRows& v, int x_dtype, int64_t n_tokens,
                             const KvPool& pool, const int64_t* slots, hipStream_t stream) {
  const int64_t es = x_dtype == kDtypeF32 ? 4 : 2, cs = pool.fp8 ? 1 : 2;
  WriteArgs a;
  const KvRows* in[2] = {&k, &v};
  void* cache[2] = {pool.k, pool.v};
  const float* scale[2] = {pool.k_scale, pool.v_scale};
  for (int i = 0; i < 2; ++i) {
    a.x[i] = static_cast<const uint8_t*>(in[i]->p);
    a.x_token[i] = in[i]->token * es;
    a.x_head[i] = in[i]->head * es;
    a.cache[i] = static_cast<uint8_t*>(cache[i]);
    a.scale[i] = scale[i];
  }
  a.page_stride = pool.page_stride * cs;
  a.head_stride = pool.head_stride * cs;
  a.token_stride = pool.token_stride * cs;
  a.slots = slots;
  a.n_slots = pool.n_pages * pool.page_size;
  const unsigned per_head = static_cast<unsigned>(pool.d / 16);
  const unsigned per_token = per_head * static_cast<unsigned>(pool.n_heads);
  a.groups = static_cast<unsigned>(n_tokens) * per_token;
  a.per_token = FastDiv::of(per_token);
  a.per_head = FastDiv::of(per_head);
  a.page = FastDiv::of(static_cast<unsigned>(pool.page_size));
  const dim3 grid((a.groups + 255u) / 256u, 2);
  if (x_dtype == kDtypeF32) {
    if (pool.fp8) page_write_kernel<0, true><<<grid, 256, 0, stream>>>(a);
    else page_write_kernel<0, false><<<grid, 256, 0, stream>>>(a);
  } else {
    if (pool.fp8) page_write_kernel<1, true><<<grid, 256, 0, stream>>>(a);
    else page_write_kernel<1, false><<<grid, 256, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
