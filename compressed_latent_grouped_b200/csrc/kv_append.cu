// Append of k / v rows to the cache with the rotary embedding of q and k on the
// way ("Compressed Convolutional Attention", Methodologie 4, for the rotation;
// Probleemstelling 2: the cache grows with the sequence), into a cache in the
// working type or in 8 bits with one scale per block of tokens and kv head, and
// the read of cached rows back as values.
//
// Rotation: pair (i, i + d/2) of position p turns by p theta_i.  The angle is a
// 0.64 fixed-point fraction of a turn, p * frac_i modulo 2^64, which reduces it
// exactly at any position; a CTA computes each (token, pair) cosine and sine
// once, in shared memory, for all its q and k heads, because at two bytes per
// element a sine per head would cost more than the memory traffic.
//
// 8-bit blocks: value = code * scale, scale = max(held scale, amax of the new
// rows / qmax).  One CTA owns one block of one kv head, k or v: it keeps the
// block's rotated rows as fp32 in shared memory, reduces their amax, rounds
// again the codes that earlier calls stored if the scale grew, and writes the
// new codes.  Nothing else writes that block, so no atomics are needed and the
// result does not depend on the schedule.
//
// Bound: memory.  Every row is read once and written once.
#include "cache_codes.cuh"

namespace ccgqa {
namespace {

constexpr int kAppThreads = 256;
constexpr float kTurn = 5.42101086242752217e-20f;   // 2^-64

template <typename T>
struct Vec16 {
  static constexpr int N = 16 / sizeof(T);
  T v[N];
};
template <typename T>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[16 / sizeof(T)]) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const T* t = reinterpret_cast<const T*>(&r);
#pragma unroll
  for (int i = 0; i < static_cast<int>(16 / sizeof(T)); ++i) x[i] = to_f32(t[i]);
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[16 / sizeof(T)]) {
  uint4 r;
  T* t = reinterpret_cast<T*>(&r);
#pragma unroll
  for (int i = 0; i < static_cast<int>(16 / sizeof(T)); ++i) t[i] = from_f32<T>(x[i]);
  *reinterpret_cast<uint4*>(p) = r;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Length and number of new rows of sequence b; false when the sequence is
// skipped (the first thread of one CTA per sequence reports why).
template <typename T>
__device__ __forceinline__ bool seq_span(const AppendArgs<T>& a, int b, bool report, int* L, int* nv) {
  *L = a.len[b];
  *nv = a.n_valid ? a.n_valid[b] : a.n_new;
  int bit = 0;
  if (*nv < 0 || *nv > a.n_new) bit = CCGQA_DEVERR_INDEX;
  else if (*L < 0 || static_cast<int64_t>(*L) + *nv > a.cap) bit = CCGQA_DEVERR_CAPACITY;
  if (bit && report) raise_dev_err(a.dev_err, bit);
  return bit == 0;
}

__device__ __forceinline__ float2 turn(int64_t pos, uint64_t frac) {
  const uint64_t ph = static_cast<uint64_t>(pos) * frac;
  float s, c;
  sincospif(2.0f * (static_cast<float>(static_cast<int64_t>(ph)) * kTurn), &s, &c);
  return make_float2(c, s);
}

// Rows of tokens [i0, i0 + tt): q (rotated) and, for a cache in the working
// type, k (rotated) and v.
template <typename T, bool kKv>
__device__ __forceinline__ void append_rows(const AppendArgs<T>& a, int b, int L, int nv, int i0, float2* cs) {
  constexpr int V = Vec16<T>::N;
  const int half = a.d >> 1, nch = half / V;
  const int tt = min(a.tile_tokens, nv - i0);
  const int64_t p0 = (a.pos ? a.pos[b] : L) + static_cast<int64_t>(i0);
  if (a.rope_on)
    for (int x = threadIdx.x; x < tt * half; x += kAppThreads)
      cs[x] = turn(p0 + x / half, a.rope_frac[x % half]);
  __syncthreads();
  const int n_q = a.q.ptr ? a.Hq : 0;
  const int heads = n_q + (kKv ? 2 * a.Hkv : 0);
  for (int x = threadIdx.x; x < tt * heads * nch; x += kAppThreads) {
    const int c = x % nch, hh = (x / nch) % heads, i = x / (nch * heads);
    const bool is_q = hh < n_q, is_k = !is_q && hh < n_q + a.Hkv;
    const int h = is_q ? hh : (is_k ? hh - n_q : hh - n_q - a.Hkv);
    const Rows& src = is_q ? a.q : (is_k ? a.k : a.v);
    const T* p = static_cast<const T*>(src.ptr) + b * src.batch + (i0 + i) * src.token +
                 h * src.head + c * V;
    float lo[V], hi[V];
    load_vec(p, lo);
    load_vec(p + half, hi);
    if (a.rope_on && (is_q || is_k)) {
      const float2* t = cs + i * half + c * V;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float x0 = lo[e], x1 = hi[e];
        lo[e] = x0 * t[e].x - x1 * t[e].y;
        hi[e] = x0 * t[e].y + x1 * t[e].x;
      }
    }
    if (is_q || (is_k && a.k_out.ptr)) {
      const Rows& dst = is_q ? a.q_out : a.k_out;
      T* o = static_cast<T*>(dst.ptr) + b * dst.batch + (i0 + i) * dst.token + h * dst.head + c * V;
      store_vec(o, lo);
      store_vec(o + half, hi);
    }
    if (!is_q) {
      const int64_t row = kv_row(a.pages, b, h, a.Hkv, a.cap, static_cast<int64_t>(L) + i0 + i);
      if (row < 0) {
        raise_dev_err(a.dev_err, CCGQA_DEVERR_INDEX);
      } else {
        T* o = static_cast<T*>(is_k ? a.ck : a.cv) + row * a.d + c * V;
        store_vec(o, lo);
        store_vec(o + half, hi);
      }
    }
  }
}

// One 8-bit block (token block j of kv head g, k or v).
template <typename T, int FMT>
__device__ __forceinline__ void append_block(const AppendArgs<T>& a, int b, int L, int nv, int jj, int g, bool is_k,
                                             float* stash) {
  constexpr int V = Vec16<T>::N;
  __shared__ float red[kAppThreads / 32];
  const int blk = 1 << a.block_shift;
  const int64_t t0 = (static_cast<int64_t>(L >> a.block_shift) + jj) << a.block_shift;
  const int r0 = max(static_cast<int>(L - t0), 0);                 // first new row of the block
  const int64_t end = static_cast<int64_t>(L) + nv - t0;
  const int r1 = end < blk ? static_cast<int>(end) : blk;          // past its last new row
  if (r1 <= r0) return;
  const int d = a.d, half = d >> 1, nch = half / V;
  const Rows& src = is_k ? a.k : a.v;
  const T* base = static_cast<const T*>(src.ptr) + b * src.batch + g * src.head;
  const int64_t i0 = t0 - L;                                       // new row index of block row 0
  const int64_t p0 = (a.pos ? a.pos[b] : L) + i0;
  const bool rot = is_k && a.rope_on;
  float amax = 0.f;
  for (int x = threadIdx.x; x < (r1 - r0) * nch; x += kAppThreads) {
    const int c = x % nch, r = r0 + x / nch;
    const T* p = base + (i0 + r) * src.token + c * V;
    float lo[V], hi[V];
    load_vec(p, lo);
    load_vec(p + half, hi);
    if (rot) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float2 t = turn(p0 + r, a.rope_frac[c * V + e]);
        const float x0 = lo[e], x1 = hi[e];
        lo[e] = x0 * t.x - x1 * t.y;
        hi[e] = x0 * t.y + x1 * t.x;
      }
    }
    float* s = stash + r * d + c * V;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      amax = max_nan(amax, max_nan(fabsf(lo[e]), fabsf(hi[e])));
      s[e] = lo[e];
      s[half + e] = hi[e];
    }
    if (is_k && a.k_out.ptr) {
      T* o = static_cast<T*>(a.k_out.ptr) + b * a.k_out.batch + (i0 + r) * a.k_out.token +
             g * a.k_out.head + c * V;
      store_vec(o, lo);
      store_vec(o + half, hi);
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = red[0];
#pragma unroll
  for (int w = 1; w < kAppThreads / 32; ++w) amax = max_nan(amax, red[w]);
  const int64_t row0 = kv_row(a.pages, b, g, a.Hkv, a.cap, t0);
  if (row0 < 0) {
    if (threadIdx.x == 0) raise_dev_err(a.dev_err, CCGQA_DEVERR_INDEX);
    return;
  }
  // rows are in whole blocks everywhere, so a block's scale index is its row / block
  float* scale = (is_k ? a.k_scale : a.v_scale) + (row0 >> a.block_shift);
  constexpr float kMaxCode = FMT == kCacheI8 ? 127.0f : 448.0f;
  const float s_old = r0 > 0 ? *scale : 0.f;
  const float s_new = max_nan(s_old, amax / kMaxCode);
  const float by = s_new == 0.f ? 1.0f : s_new;   // a block of zeros keeps scale 0
  __syncthreads();   // every thread has read the held scale
  if (threadIdx.x == 0) *scale = s_new;
  uint8_t* codes = static_cast<uint8_t*>(is_k ? a.ck : a.cv) + row0 * d;
  const int n8 = d >> 3;
  if (s_new > s_old && r0 > 0) {
    const float ratio = s_old / s_new;
    for (int x = threadIdx.x; x < r0 * n8; x += kAppThreads) {
      uint2* w = reinterpret_cast<uint2*>(codes + x * 8);
      float v[8];
      decode8<FMT>(*w, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= ratio;
      *w = encode8<FMT>(v);
    }
  }
  for (int x = threadIdx.x; x < (r1 - r0) * n8; x += kAppThreads) {
    const float* s = stash + r0 * d + x * 8;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = s[e] / by;
    *reinterpret_cast<uint2*>(codes + r0 * d + x * 8) = encode8<FMT>(v);
  }
}

// CTAs [0, n_blocks): the 8-bit blocks; the rest: tiles of tokens for the rows
// stored in the working type.  With tickets, the last CTA of a sequence to have
// read its length moves it on; which one that is does not show in any result.
template <typename T, int FMT>
__global__ void __launch_bounds__(kAppThreads)
    append_kernel(const __grid_constant__ AppendArgs<T> a, int n_blocks, int per_seq, int tiles, int ctas_per_seq) {
  pdl_enter();
  extern __shared__ __align__(16) uint8_t smem[];
  const int x = blockIdx.x;
  const bool block = FMT != 0 && x < n_blocks;
  const int in_seq = block ? per_seq * a.Hkv * 2 : tiles;   // CTAs of this kind per sequence
  const int y = block ? x : x - n_blocks;
  const int b = y / in_seq, i = y % in_seq;
  int L, nv;
  const bool ok = seq_span(a, b, i == 0 && (block || n_blocks == 0) && threadIdx.x == 0, &L, &nv);
  if (a.tickets) {
    __syncthreads();   // every thread of this CTA holds the length
    if (threadIdx.x == 0) {
      __threadfence();
      if (atomicAdd(a.tickets + b, 1) == ctas_per_seq - 1) {
        a.tickets[b] = 0;
        if (ok) a.len[b] = L + nv;
      }
    }
  }
  if (!ok) return;
  if constexpr (FMT != 0) {
    if (block) {
      append_block<T, FMT>(a, b, L, nv, i / 2 / a.Hkv, i / 2 % a.Hkv, (i & 1) == 0, reinterpret_cast<float*>(smem));
      return;
    }
  }
  append_rows<T, FMT == 0>(a, b, L, nv, i * a.tile_tokens, reinterpret_cast<float2*>(smem));
}

template <typename T>
__global__ void __launch_bounds__(128) bump_kernel(const __grid_constant__ AppendArgs<T> a) {
  pdl_enter();
  const int b = blockIdx.x * 128 + threadIdx.x;
  int L, nv;
  if (b < a.B && seq_span(a, b, false, &L, &nv)) a.len[b] = L + nv;
}

template <typename T, int FMT>
cudaError_t launch_append_fmt(AppendArgs<T> a, cudaStream_t stream) {
  const int half = a.d / 2;
  a.tile_tokens = kAppThreads / half > 0 ? kAppThreads / half : 1;
  const int tiles = (a.n_new + a.tile_tokens - 1) / a.tile_tokens;
  const bool rows = FMT == 0 || a.q.ptr;
  const int64_t n_rows = rows ? static_cast<int64_t>(a.B) * tiles : 0;
  const int blk = 1 << a.block_shift;
  // a run of n_new tokens that starts anywhere in a block touches this many blocks
  const int per_seq = FMT == 0 ? 1 : (a.n_new + 2 * blk - 2) / blk;
  const int64_t n_blocks = FMT == 0 ? 0 : static_cast<int64_t>(a.B) * per_seq * a.Hkv * 2;
  if (n_rows + n_blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const int ctas_per_seq = static_cast<int>((n_rows + n_blocks) / a.B);
  size_t smem = static_cast<size_t>(a.tile_tokens) * half * sizeof(float2);
  if (FMT != 0 && static_cast<size_t>(blk) * a.d * 4 > smem) smem = static_cast<size_t>(blk) * a.d * 4;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(append_kernel<T, FMT>), static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  e = launch_pdl(append_kernel<T, FMT>, dim3(static_cast<unsigned>(n_rows + n_blocks)), dim3(kAppThreads),
                 smem, stream, a, static_cast<int>(n_blocks), per_seq, tiles, ctas_per_seq);
  if (e != cudaSuccess) return e;
  count_launches(1);
  if (!a.tickets) {
    e = launch_pdl(bump_kernel<T>, dim3((a.B + 127) / 128), dim3(128), 0, stream, a);
    if (e != cudaSuccess) return e;
    count_launches(1);
  }
  return cudaGetLastError();
}

// ----------------------------------------------------------------- read back
template <typename T, int FMT>
__global__ void __launch_bounds__(kAppThreads)
    kv_read_kernel(const __grid_constant__ ReadArgs a, int64_t total) {
  pdl_enter();
  constexpr int V = 8;
  const int nch = a.d / V;
  for (int64_t x = static_cast<int64_t>(blockIdx.x) * kAppThreads + threadIdx.x; x < total;
       x += static_cast<int64_t>(gridDim.x) * kAppThreads) {
    const int c = static_cast<int>(x % nch);
    int64_t y = x / nch;
    const int i = static_cast<int>(y % a.n);   // tokens of a head are neighbours in the cache
    y /= a.n;
    const int g = static_cast<int>(y % a.Hkv), b = static_cast<int>(y / a.Hkv);
    const int L = a.len[b];
    if (L < 0 || L > a.cap) {
      if (i == 0 && g == 0 && c == 0) raise_dev_err(a.dev_err, CCGQA_DEVERR_CAPACITY);
      continue;
    }
    const int64_t t = static_cast<int64_t>(a.first) + i;
    if (t >= L) continue;
    const int64_t row = kv_row(a.pages, b, g, a.Hkv, a.cap, t);
    if (row < 0) {
      raise_dev_err(a.dev_err, CCGQA_DEVERR_INDEX);
      continue;
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const Rows& dst = w ? a.v_out : a.k_out;
      T* o = static_cast<T*>(dst.ptr) + b * dst.batch + i * dst.token + g * dst.head + c * V;
      if constexpr (FMT == 0) {
        const uint4* s = reinterpret_cast<const uint4*>(static_cast<const T*>(w ? a.cv : a.ck) + row * a.d + c * V);
#pragma unroll
        for (int u = 0; u < static_cast<int>(V * sizeof(T) / 16); ++u) reinterpret_cast<uint4*>(o)[u] = s[u];
      } else {
        float v[8];
        decode8<FMT>(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(w ? a.cv : a.ck) + row * a.d + c * V), v);
        const float s = (w ? a.v_scale : a.k_scale)[row >> a.block_shift];
        float f[16 / sizeof(T)];
#pragma unroll
        for (int u = 0; u < static_cast<int>(V * sizeof(T) / 16); ++u) {
#pragma unroll
          for (int e = 0; e < static_cast<int>(16 / sizeof(T)); ++e) f[e] = v[u * (16 / sizeof(T)) + e] * s;
          store_vec(o + u * (16 / sizeof(T)), f);
        }
      }
    }
  }
}

template <typename T, int FMT>
cudaError_t launch_read_fmt(const ReadArgs& a, cudaStream_t stream) {
  const int64_t total = static_cast<int64_t>(a.B) * a.Hkv * a.n * (a.d / 8);
  const int64_t want = (total + kAppThreads - 1) / kAppThreads;
  const int64_t most = static_cast<int64_t>(sm_count()) * 64;
  const cudaError_t e = launch_pdl(kv_read_kernel<T, FMT>, dim3(static_cast<unsigned>(want < most ? want : most)),
                                   dim3(kAppThreads), 0, stream, a, total);
  if (e != cudaSuccess) return e;
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

template <typename T>
cudaError_t launch_append_rope(const AppendArgs<T>& a, int fmt, cudaStream_t stream) {
  switch (fmt) {
    case 0: return launch_append_fmt<T, 0>(a, stream);
    case kCacheI8: return launch_append_fmt<T, kCacheI8>(a, stream);
    case kCacheE4M3: return launch_append_fmt<T, kCacheE4M3>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}
template cudaError_t launch_append_rope<float>(const AppendArgs<float>&, int, cudaStream_t);
template cudaError_t launch_append_rope<bf16>(const AppendArgs<bf16>&, int, cudaStream_t);

template <typename T>
cudaError_t launch_kv_read(const ReadArgs& a, int fmt, cudaStream_t stream) {
  switch (fmt) {
    case 0: return launch_read_fmt<T, 0>(a, stream);
    case kCacheI8: return launch_read_fmt<T, kCacheI8>(a, stream);
    case kCacheE4M3: return launch_read_fmt<T, kCacheE4M3>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}
template cudaError_t launch_kv_read<float>(const ReadArgs&, int, cudaStream_t);
template cudaError_t launch_kv_read<bf16>(const ReadArgs&, int, cudaStream_t);

}  // namespace ccgqa
