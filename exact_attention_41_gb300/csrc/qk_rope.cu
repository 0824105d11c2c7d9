// Per-head RMS norm and position rotation of queries and keys in one pass,
// its gradient, and the append of keys and values to a paged cache with both
// on the way.  (The source pages have no counterpart: they start at q, k, v.)
//
//   xh = x / sqrt(mean(x^2) + eps),  z = w xh,  y = R(pos) z
//   R(pos): pair j of the first `rot` elements turns by pos f_j; pairs are
//   (j, j + rot/2), or (2j, 2j + 1) when interleaved
//
// and backwards, with gz = R(-pos) gy:
//
//   gw = sum over rows and heads of gz xh
//   gx = (gz w - xh mean(gz w xh)) / sqrt(mean(x^2) + eps)
//
// Angles.  f_j comes as the fraction of a full turn per position, in units of
// 2^-64 turns, so position * phase in 64-bit integers wraps exactly at whole
// turns: no position is far enough to lose the angle, and no 64-bit
// floating-point unit is needed.
//
// Layout.  A thread holds 16 elements of one head as two 16-byte pieces: the
// two halves of eight rotation pairs (or eight interleaved pairs).  Its eight
// cosines and sines are then the same for every head of the token, and a head
// is D / 16 neighbouring lanes, so the norm's sum is log2(D / 16) shuffles.
// Everything is held in fp32 and rounded once, to the output.
#include "kernels.h"

namespace attn {
namespace {

constexpr int kWarps = 4;       // warps of a forward or append block
constexpr int kBwdWarps = 8;    // warps of a backward block

// Where the 16 elements of thread `t` of a head sit: elements 0-7 at o0, 8-15
// at o1.
struct Slots {
  int o0, o1;
  bool turn;  // the elements are rotation pairs
};
__device__ __forceinline__ Slots slots_of(int t, int rot, int interleaved) {
  const bool turn = 16 * t < rot;
  if (turn && !interleaved) return {8 * t, rot / 2 + 8 * t, true};
  return {16 * t, 16 * t + 8, turn};
}

template <typename T>
__device__ __forceinline__ void load16(const T *row, const Slots &sl, float (&x)[16]) {
  load_vec<T, 8>(row + sl.o0, x);
  load_vec<T, 8>(row + sl.o1, x + 8);
}
template <typename T>
__device__ __forceinline__ void store16(T *row, const Slots &sl, const float (&x)[16]) {
  store_vec<T, 8>(row + sl.o0, x);
  store_vec<T, 8>(row + sl.o1, x + 8);
}

// cos and sin of the eight pairs 8t .. 8t+7 at position `pos`.
__device__ __forceinline__ void angles(const uint64_t *phases, int t, int64_t pos, float (&c)[8],
                                       float (&s)[8]) {
  const ulonglong2 *p = reinterpret_cast<const ulonglong2 *>(phases + 8 * t);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const ulonglong2 f = p[e];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // turns mod 1 in 2^-64, rounded to 2^-32 of a turn = 2^-31 of a half turn
      const uint64_t turn = (uint64_t)pos * (u ? f.y : f.x) + 0x80000000ull;
      const float half_turns = (float)(int32_t)(turn >> 32) * 4.656612873077393e-10f;  // 2^-31
      sincospif(half_turns, &s[2 * e + u], &c[2 * e + u]);
    }
  }
}

// Turns the pairs of x by the angles (sign = 1) or back (sign = -1).
__device__ __forceinline__ void rotate(float (&x)[16], const float (&c)[8], const float (&s)[8],
                                       float sign, int interleaved) {
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = x[2 * e], b = x[2 * e + 1], sn = sign * s[e];
      x[2 * e] = a * c[e] - b * sn;
      x[2 * e + 1] = a * sn + b * c[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = x[e], b = x[8 + e], sn = sign * s[e];
      x[e] = a * c[e] - b * sn;
      x[8 + e] = a * sn + b * c[e];
    }
  }
}

// Sum over the D / 16 lanes of a head.
template <int D>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = 1; o < D / 16; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int D>
__device__ __forceinline__ float inv_rms(const float (&x)[16], float eps) {
  float q = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) q = fmaf(x[e], x[e], q);
  return rsqrtf(head_sum<D>(q) * (1.f / D) + eps);
}

// Cache rows of token `r`, or nullptr where the token is not to be written.
struct Token {
  int64_t pos;
  bool live;       // a row of some sequence
  bool cached;     // its cache slot is valid
  int64_t page;
  int slot;
};

// Sequence, position and cache slot of packed row `r`.  Whole warp.
__device__ __forceinline__ Token find_token(const RopeArgs &a, int r) {
  const int lane = threadIdx.x & 31;
  Token tk{0, false, false, 0, 0};
  // sequence = how many sequences end at or before r
  int seq = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const bool ended = b0 + lane < a.batch && a.cu_seqlens[b0 + lane + 1] <= r;
    seq += __popc(__ballot_sync(0xffffffffu, ended));
  }
  if (seq >= a.batch) return tk;  // behind the last sequence
  const int first = a.cu_seqlens[seq];
  const int cached = a.cache_seqlens[seq];
  if (first < 0 || r < first || cached < 0) {
    if (lane == 0) raise_error(a.err, kErrBadSeqlen);
    return tk;
  }
  tk.live = true;
  tk.pos = (int64_t)cached + (r - first);
  const int64_t pg = tk.pos / a.page_size;
  if (pg >= a.max_pages) {
    if (lane == 0) raise_error(a.err, kErrCacheOverflow);
    return tk;
  }
  const int page = a.block_table ? a.block_table[(int64_t)seq * a.max_pages + pg] : seq;
  if (page < 0 || page >= a.num_pages) {
    if (lane == 0) raise_error(a.err, kErrPageOutOfRange);
    return tk;
  }
  tk.cached = true;
  tk.page = page;
  tk.slot = (int)(tk.pos - pg * a.page_size);
  return tk;
}

// One warp takes every `parts`-th group of 32 / (D / 16) heads of one token:
// first the query heads, then the key heads, then (append) the value heads.
template <typename T, int D, bool kAppend>
__global__ void __launch_bounds__(kWarps * 32) norm_rope_kernel(const RopeArgs a) {
  constexpr int LPH = D / 16, HPW = 32 / LPH;
  const int lane = threadIdx.x & 31, t = lane % LPH, sub = lane / LPH;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t row = unit / a.parts;
  if (row >= a.rows) return;
  const int part = (int)(unit % a.parts);
  int64_t pos;
  T *kd = nullptr, *vd = nullptr;
  if constexpr (kAppend) {
    const Token tk = find_token(a, (int)row);
    if (!tk.live) return;
    pos = tk.pos;
    if (tk.cached) {
      const int64_t in_page = (int64_t)tk.slot * a.hkv * D;
      kd = static_cast<T *>(a.k_out) + tk.page * a.k_out_rs + in_page;
      vd = static_cast<T *>(a.v_out) + tk.page * a.v_out_rs + in_page;
    }
  } else {
    pos = a.positions ? a.positions[row] : row % a.s;
    kd = static_cast<T *>(a.k_out) + row * a.k_out_rs;
  }
  T *qd = static_cast<T *>(a.q_out) + row * a.q_out_rs;
  const T *qs = static_cast<const T *>(a.q) + row * a.q_rs;
  const T *ks = static_cast<const T *>(a.k) + row * a.k_rs;
  const Slots sl = slots_of(t, a.rot, a.interleaved);
  float c[8], s[8];
  if (sl.turn) angles(a.phases, t, pos, c, s);
  const int nq = (a.hq + HPW - 1) / HPW, nk = (a.hkv + HPW - 1) / HPW;
  const int n = nq + nk * (kAppend ? 2 : 1);
  for (int it = part; it < n; it += a.parts) {
    if (kAppend && it >= nq + nk) {  // values: copied
      const int h = (it - nq - nk) * HPW + sub;
      if (h < a.hkv && vd) {
        const T *src = static_cast<const T *>(a.v) + row * a.v_rs + h * D + 16 * t;
        uint4 *dst = reinterpret_cast<uint4 *>(vd + h * D + 16 * t);
        dst[0] = reinterpret_cast<const uint4 *>(src)[0];
        dst[1] = reinterpret_cast<const uint4 *>(src)[1];
      }
      continue;
    }
    const bool is_q = it < nq;
    const int h = (is_q ? it : it - nq) * HPW + sub;
    const bool on = h < (is_q ? a.hq : a.hkv);
    const T *src = (is_q ? qs : ks) + h * D;
    T *dst = is_q ? qd : kd;
    const T *w = static_cast<const T *>(is_q ? a.q_weight : a.k_weight);
    float x[16];
    if (on) {
      load16(src, sl, x);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = 0.f;
    }
    if (w) {
      const float r = inv_rms<D>(x, a.eps);
      float wv[16];
      load16(w, sl, wv);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = x[e] * r * wv[e];
    }
    if (sl.turn) rotate(x, c, s, 1.f, a.interleaved);
    if (on && (!kAppend || dst)) store16(dst + h * D, sl, x);
  }
}

// Gradient of one head's norm and rotation; adds the weight's gradient.
template <typename T, int D>
__device__ __forceinline__ void bwd_head(const T *x_row, const T *gy_row, T *gx_row, bool on,
                                         const T *w, float eps, const Slots &sl,
                                         const float (&c)[8], const float (&s)[8],
                                         int interleaved, float (&gw)[16]) {
  float g[16], x[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) g[e] = x[e] = 0.f;
  if (on) {
    load16(gy_row, sl, g);
    if (w) load16(x_row, sl, x);
  }
  if (sl.turn) rotate(g, c, s, -1.f, interleaved);
  if (w) {
    float wv[16];
    load16(w, sl, wv);
    const float r = inv_rms<D>(x, eps);
    float dot = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      x[e] *= r;
      gw[e] = fmaf(g[e], x[e], gw[e]);
      g[e] *= wv[e];
      dot = fmaf(g[e], x[e], dot);
    }
    dot = head_sum<D>(dot) * (1.f / D);
#pragma unroll
    for (int e = 0; e < 16; ++e) g[e] = (g[e] - x[e] * dot) * r;
  }
  if (on) store16(gx_row, sl, g);
}

// Persistent: a warp takes every (blocks * kBwdWarps)-th token and keeps the
// weights' gradients of its tokens in registers; the block adds its warps in
// order and writes one partial per weight, which a second kernel adds in
// order, so the result does not change from run to run.
template <typename T, int D>
__global__ void __launch_bounds__(kBwdWarps * 32) norm_rope_bwd_kernel(const RopeArgs a) {
  constexpr int LPH = D / 16, HPW = 32 / LPH;
  __shared__ float part[kBwdWarps][2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane % LPH, sub = lane / LPH;
  const Slots sl = slots_of(t, a.rot, a.interleaved);
  float gwq[16], gwk[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) gwq[e] = gwk[e] = 0.f;
  for (int64_t row = (int64_t)blockIdx.x * kBwdWarps + warp; row < a.rows;
       row += (int64_t)gridDim.x * kBwdWarps) {
    const int64_t pos = a.positions ? a.positions[row] : row % a.s;
    float c[8], s[8];
    if (sl.turn) angles(a.phases, t, pos, c, s);
    for (int h = sub; h - sub < a.hq; h += HPW)
      bwd_head<T, D>(static_cast<const T *>(a.q) + row * a.q_rs + h * D,
                     static_cast<const T *>(a.gq) + row * a.gq_rs + h * D,
                     static_cast<T *>(a.q_out) + row * a.q_out_rs + h * D, h < a.hq,
                     static_cast<const T *>(a.q_weight), a.eps, sl, c, s, a.interleaved, gwq);
    for (int h = sub; h - sub < a.hkv; h += HPW)
      bwd_head<T, D>(static_cast<const T *>(a.k) + row * a.k_rs + h * D,
                     static_cast<const T *>(a.gk) + row * a.gk_rs + h * D,
                     static_cast<T *>(a.k_out) + row * a.k_out_rs + h * D, h < a.hkv,
                     static_cast<const T *>(a.k_weight), a.eps, sl, c, s, a.interleaved, gwk);
  }
  if (!a.q_weight && !a.k_weight) return;
  // the HPW heads of a warp, then its warps
#pragma unroll
  for (int e = 0; e < 16; ++e) {
#pragma unroll
    for (int o = LPH; o < 32; o <<= 1) {
      gwq[e] += __shfl_xor_sync(0xffffffffu, gwq[e], o);
      gwk[e] += __shfl_xor_sync(0xffffffffu, gwk[e], o);
    }
  }
  if (sub == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      part[warp][0][sl.o0 + e] = gwq[e];
      part[warp][0][sl.o1 + e] = gwq[8 + e];
      part[warp][1][sl.o0 + e] = gwk[e];
      part[warp][1][sl.o1 + e] = gwk[8 + e];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kBwdWarps * 32) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kBwdWarps; ++w) v += part[w][i / D][i % D];
    a.gw_part[(int64_t)blockIdx.x * 2 * D + i] = v;
  }
}

// gw = sum of the blocks' partials, in a fixed order; 32 columns a block.
template <typename T, int D>
__global__ void __launch_bounds__(1024) weight_grad_kernel(const RopeArgs a, int blocks) {
  __shared__ float sum[32][33];
  const int col = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + col;
  float v = 0.f;
  for (int b = grp; b < blocks; b += 32) v += a.gw_part[(int64_t)b * 2 * D + i];
  sum[grp][col] = v;
  __syncthreads();
  if (grp == 0) {
    float r = 0.f;
#pragma unroll
    for (int g = 0; g < 32; ++g) r += sum[g][col];
    T *dst = static_cast<T *>(i < D ? a.q_gw : a.k_gw);
    if (dst) dst[i % D] = Elem<T>::from_f(r);
  }
}

template <typename T, int D>
cudaError_t fwd(RopeArgs a, int sms, cudaStream_t st) {
  constexpr int HPW = 32 / (D / 16);
  const bool append = a.cu_seqlens != nullptr;
  const int n = (a.hq + HPW - 1) / HPW + (a.hkv + HPW - 1) / HPW * (append ? 2 : 1);
  if (n == 0) return cudaSuccess;
  // few tokens: a token's head groups go to separate warps
  a.parts = 1;
  while (a.parts < n && (int64_t)a.rows * a.parts < (int64_t)sms * 32) a.parts *= 2;
  a.parts = a.parts < n ? a.parts : n;
  const int64_t grid = ((int64_t)a.rows * a.parts + kWarps - 1) / kWarps;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  debug_log("%s: norm_rope_kernel d=%d, %d tokens x %d warps each, grid=%lld", append ? "append" : "norm+rotation",
            D, a.rows, a.parts, (long long)grid);
  if (append)
    norm_rope_kernel<T, D, true><<<(unsigned)grid, kWarps * 32, 0, st>>>(a);
  else
    norm_rope_kernel<T, D, false><<<(unsigned)grid, kWarps * 32, 0, st>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t bwd(const RopeArgs &a, int sms, cudaStream_t st) {
  const int64_t want = ((int64_t)a.rows + kBwdWarps - 1) / kBwdWarps;
  const int blocks = (int)(want < rope_bwd_blocks(sms) ? want : rope_bwd_blocks(sms));
  debug_log("norm+rotation backward: norm_rope_bwd_kernel d=%d, %d tokens, grid=%d", D, a.rows, blocks);
  if (blocks > 0) {  // no tokens: the weights' gradients are empty sums
    norm_rope_bwd_kernel<T, D><<<blocks, kBwdWarps * 32, 0, st>>>(a);
    count_launches(1);
  }
  if (a.q_weight || a.k_weight) {
    weight_grad_kernel<T, D><<<2 * D / 32, 1024, 0, st>>>(a, blocks);
    count_launches(1);
  }
  return cudaGetLastError();
}

}  // namespace

int rope_bwd_blocks(int sms) { return 3 * sms; }

cudaError_t launch_norm_rope(const RopeArgs &a, int sms, cudaStream_t st) {
  const bool bf = a.dtype == ATTN_BF16;
  switch (a.d) {
    case 64: return bf ? fwd<__nv_bfloat16, 64>(a, sms, st) : fwd<__half, 64>(a, sms, st);
    case 128: return bf ? fwd<__nv_bfloat16, 128>(a, sms, st) : fwd<__half, 128>(a, sms, st);
    case 256: return bf ? fwd<__nv_bfloat16, 256>(a, sms, st) : fwd<__half, 256>(a, sms, st);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_norm_rope_bwd(const RopeArgs &a, int sms, cudaStream_t st) {
  const bool bf = a.dtype == ATTN_BF16;
  switch (a.d) {
    case 64: return bf ? bwd<__nv_bfloat16, 64>(a, sms, st) : bwd<__half, 64>(a, sms, st);
    case 128: return bf ? bwd<__nv_bfloat16, 128>(a, sms, st) : bwd<__half, 128>(a, sms, st);
    case 256: return bf ? bwd<__nv_bfloat16, 256>(a, sms, st) : bwd<__half, 256>(a, sms, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace attn
