// RMS norm of every query and key head and the rotary position embedding, in one pass, forward and
// backward.
//
// Forward, for each token t and head: with r = 1 / sqrt(mean(x^2) + eps), z = x r w (w: the query or
// key weight of d elements; without weights z = x), and for each rotated pair i of elements
//     y_a = z_a cos(phi) - z_b sin(phi),  y_b = z_b cos(phi) + z_a sin(phi),
//     phi = positions[axis(i)][t] inv_freq[i]
// Backward: g = the inverse rotation of dy, then with xhat = x r
//     dw = sum over tokens and heads of g xhat,  dx = r (g w - xhat mean(g w xhat)).
//
// Bound by HBM: every element is read once and written once (backward: two reads). A group of d / 16
// lanes holds one head, 16 elements a lane, chosen so that both members of each pair are in the same
// lane: the rotation needs no exchange between lanes, the norm three or two shuffles, and a warp
// takes 4 heads (d = 128) or 8 (d = 64) at once with 16-byte accesses. A warp's angles are computed
// once per token and kept in registers for all of its heads.
//
// Angles: positions reach far beyond the 24 bits of an fp32 product, so the turn phi / 2 pi is formed
// in 64-bit fixed point, where the multiplication drops whole turns by itself: inv_freq / 2 pi becomes
// a fraction of 2^64 once per thread (in fp64), and position times fraction mod 2^64 is exact.
// Norms, weights' gradients and products are fp32; a result is rounded to bf16 once, at the end.
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>
#include <cstring>
#include "../../include/fa.h"
#include "host.cuh"
#include "kernels.cuh"

namespace fa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kMaxAxes = 4;

struct RopeParams {
  // [0] queries, [1] keys; strides between tokens in elements
  const uint16_t* x[2];
  const uint16_t* dy[2];   // backward
  uint16_t* out[2];        // forward: y, backward: dx
  int64_t x_stride[2], dy_stride[2], out_stride[2];
  const uint16_t* w[2];    // bf16 weights of d elements, or null: no norm
  const int32_t* positions;  // [axes, T]
  const float* inv_freq;     // [rot / 2]
  float* partial;            // backward with weights: [gridDim.x, 2, d] sums of the weights' gradients
  int64_t T;
  int heads[2], passes[2];  // passes: warp steps that cover the heads of one token
  int rot, section_end[kMaxAxes - 1];  // pairs [section_end[a - 1], section_end[a]) belong to axis a
  int parts, per_part;     // a token's passes are split over `parts` warps, `per_part` each
  float eps;
};

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

__device__ __forceinline__ void unpack8(uint4 v, float* f) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf_lo(u[i]);
    f[2 * i + 1] = bf_hi(u[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Sum over the kLanes lanes that share a head.
template <int kLanes>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int D, bool BWD, bool NORM, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kLanes = D / 16;       // lanes per head
  constexpr int kHeads = 32 / kLanes;  // heads per warp step
  __shared__ float2 angles[kRopeWarps][D / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = lane % kLanes, head_of = lane / kLanes;
  // This lane's elements: two runs of 8. Split halves: run 0 of the first half of the rotated
  // elements, run 1 the partners in the second half (past them, 16 in a row); adjacent pairs: 16 in a row.
  const int rot_lanes = p.rot / 16;
  const bool rotated = j < rot_lanes;
  int c0 = 16 * j, c1 = 16 * j + 8;
  if (!INTERLEAVED && rotated) {
    c0 = 8 * j;
    c1 = p.rot / 2 + 8 * j;
  }
  // the pairs whose angles this lane computes: lane and lane + 32
  uint64_t turn[2] = {0, 0};
  int axis[2] = {0, 0};
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int i = lane + 32 * x;
    if (i < p.rot / 2) {
      const double f = (double)p.inv_freq[i] * 0.15915494309189533577;
      turn[x] = (uint64_t)((f - floor(f)) * 18446744073709551616.0);
#pragma unroll
      for (int a = 0; a < kMaxAxes - 1; ++a) axis[x] += i >= p.section_end[a];
    }
  }
  uint4 wv[2][2];  // the lane's weights
  if constexpr (NORM) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      wv[x][0] = *reinterpret_cast<const uint4*>(p.w[x] + c0);
      wv[x][1] = *reinterpret_cast<const uint4*>(p.w[x] + c1);
    }
  }
  float dw[2][16];  // backward: this lane's share of the weights' gradients
#pragma unroll
  for (int i = 0; i < 16; ++i) dw[0][i] = dw[1][i] = 0.f;

  const int64_t units = p.T * p.parts, stride = (int64_t)gridDim.x * kRopeWarps;
  for (int64_t unit = (int64_t)blockIdx.x * kRopeWarps + warp; unit < units; unit += stride) {
    const int64_t t = unit / p.parts;
    const int first = (int)(unit % p.parts) * p.per_part;
    const int last = min(first + p.per_part, p.passes[0] + p.passes[1]);
    float cs[8], sn[8];
    if (p.rot > 0) {
      __syncwarp();  // the previous token's angles have been read
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int i = lane + 32 * x;
        if (i < p.rot / 2) {
          const int64_t pos = p.positions[axis[x] * p.T + t];
          const int32_t turns = (int32_t)(((uint64_t)pos * turn[x]) >> 32);  // 2^-32 of a turn
          float s, c;
          sincospif((float)turns * 0x1p-31f, &s, &c);
          angles[warp][i] = make_float2(c, s);
        }
      }
      __syncwarp();
      if (rotated) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 a = angles[warp][8 * j + i];
          cs[i] = a.x;
          sn[i] = a.y;
        }
      }
    }
#pragma unroll 2
    for (int pass = first; pass < last; ++pass) {
      const int which = pass >= p.passes[0];  // 0: queries, 1: keys
      const int head = (pass - (which ? p.passes[0] : 0)) * kHeads + head_of;
      const bool live = head < (which ? p.heads[1] : p.heads[0]);
      const uint16_t* src = (which ? p.x[1] : p.x[0]) + t * (which ? p.x_stride[1] : p.x_stride[0]) + head * D;
      const uint16_t* dsrc = (which ? p.dy[1] : p.dy[0]) + t * (which ? p.dy_stride[1] : p.dy_stride[0]) + head * D;
      uint16_t* dst = (which ? p.out[1] : p.out[0]) + t * (which ? p.out_stride[1] : p.out_stride[0]) + head * D;
      float x[16], g[16];
      uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0, g0 = x0, g1 = x0;
      if (live) {
        if (NORM || !BWD) {
          x0 = __ldcs(reinterpret_cast<const uint4*>(src + c0));
          x1 = __ldcs(reinterpret_cast<const uint4*>(src + c1));
        }
        if constexpr (BWD) {
          g0 = __ldcs(reinterpret_cast<const uint4*>(dsrc + c0));
          g1 = __ldcs(reinterpret_cast<const uint4*>(dsrc + c1));
        }
      }
      unpack8(x0, x);
      unpack8(x1, x + 8);
      float w[16], r = 1.f;
      if constexpr (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
        r = rsqrtf(head_sum<kLanes>(ss) * (1.f / D) + p.eps);
        unpack8(which ? wv[1][0] : wv[0][0], w);
        unpack8(which ? wv[1][1] : wv[0][1], w + 8);
      }
      if constexpr (!BWD) {
        if constexpr (NORM) {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = x[i] * r * w[i];
        }
        if (rotated) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float& a = x[INTERLEAVED ? 2 * i : i];
            float& b = x[INTERLEAVED ? 2 * i + 1 : 8 + i];
            const float a0 = a, b0 = b;
            a = a0 * cs[i] - b0 * sn[i];
            b = b0 * cs[i] + a0 * sn[i];
          }
        }
      } else {
        unpack8(g0, g);
        unpack8(g1, g + 8);
        if (rotated) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float& a = g[INTERLEAVED ? 2 * i : i];
            float& b = g[INTERLEAVED ? 2 * i + 1 : 8 + i];
            const float a0 = a, b0 = b;
            a = a0 * cs[i] + b0 * sn[i];
            b = b0 * cs[i] - a0 * sn[i];
          }
        }
        if constexpr (NORM) {
          float inner = 0.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            x[i] *= r;
            const float v = g[i] * x[i];
            if (which) dw[1][i] += v;
            else dw[0][i] += v;
            inner = fmaf(v, w[i], inner);
          }
          inner = head_sum<kLanes>(inner) * (1.f / D);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = (g[i] * w[i] - x[i] * inner) * r;
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = g[i];
        }
      }
      if (live) {
        *reinterpret_cast<uint4*>(dst + c0) = pack8(x);
        *reinterpret_cast<uint4*>(dst + c1) = pack8(x + 8);
      }
    }
  }
  if constexpr (BWD && NORM) {
    // heads of the warp, then warps of the CTA, in a fixed order; one row of partial sums per CTA
    __shared__ float sums[kRopeWarps][2][D];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float v = dw[x][i];
#pragma unroll
        for (int o = 16; o >= kLanes; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (head_of == 0) sums[warp][x][(i < 8 ? c0 : c1 - 8) + i] = v;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kRopeThreads) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < kRopeWarps; ++k) v += sums[k][i / D][i % D];
      p.partial[(int64_t)blockIdx.x * 2 * D + i] = v;
    }
  }
}

// The weights' gradients: sums of the CTAs' rows in a fixed order. One CTA per 32 columns: its warps
// take every 8th row each, and are added in order.
__global__ void __launch_bounds__(256) rope_weight_grad_kernel(const float* partial, int rows, int d, float* dq_weight,
                                                               float* dk_weight) {
  __shared__ float sums[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float v = 0.f;
#pragma unroll 8
  for (int r = warp; r < rows; r += 8) v += partial[(int64_t)r * 2 * d + col];
  sums[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
    float total = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) total += sums[k][lane];
    (col < d ? dq_weight : dk_weight)[col % d] = total;
  }
}

// Warps per SM that the kernel is spread over.
constexpr int kRopeWarpsPerSm = 32;

int rope_max_blocks(int sm_count) { return sm_count * kRopeWarpsPerSm / kRopeWarps; }

struct RopeSplit {
  int parts, per_part, blocks;
};

// A token's passes stay in one warp when there are tokens enough to fill the GPU (its angles are then
// computed once); with few tokens they are spread over more warps, down to one pass each.
RopeSplit split_rope(int64_t T, int passes, int sm_count) {
  RopeSplit s;
  const int64_t target = (int64_t)sm_count * kRopeWarpsPerSm;
  int64_t parts = T > 0 ? (target + T - 1) / T : 1;
  if (parts > passes) parts = passes;
  if (parts < 1) parts = 1;
  s.per_part = (int)((passes + parts - 1) / parts);
  s.parts = (passes + s.per_part - 1) / s.per_part;
  const int64_t blocks = (T * s.parts + kRopeWarps - 1) / kRopeWarps;
  s.blocks = (int)(blocks < rope_max_blocks(sm_count) ? blocks : rope_max_blocks(sm_count));
  return s;
}

template <int D, bool BWD>
cudaError_t launch_rope(const RopeParams& p, int blocks, bool norm, bool interleaved, cudaStream_t stream) {
  if (norm) {
    if (interleaved) rope_kernel<D, BWD, true, true><<<blocks, kRopeThreads, 0, stream>>>(p);
    else rope_kernel<D, BWD, true, false><<<blocks, kRopeThreads, 0, stream>>>(p);
  } else {
    if (interleaved) rope_kernel<D, BWD, false, true><<<blocks, kRopeThreads, 0, stream>>>(p);
    else rope_kernel<D, BWD, false, false><<<blocks, kRopeThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

// One [T, heads, d] tensor of a call: rows of heads * d elements, `stride` elements apart.
struct Rows {
  const void* ptr;
  int64_t stride;
  int heads;
};

// Whether two such tensors share an element. Rows with the same stride may be interleaved (views of
// one fused projection): they are apart when their columns are.
bool rows_overlap(const Rows& a, const Rows& b, int64_t T, int d) {
  if (!a.ptr || !b.ptr || T <= 0) return false;
  const uint64_t wa = (uint64_t)a.heads * d * 2, wb = (uint64_t)b.heads * d * 2;
  if (!overlaps(a.ptr, (uint64_t)(T - 1) * a.stride * 2 + wa, b.ptr, (uint64_t)(T - 1) * b.stride * 2 + wb))
    return false;
  if (a.stride != b.stride) return true;
  const uint64_t s = (uint64_t)a.stride * 2;
  const uint64_t x = reinterpret_cast<uintptr_t>(a.ptr), y = reinterpret_cast<uintptr_t>(b.ptr);
  const uint64_t off = y >= x ? (y - x) % s : (s - (x - y) % s) % s;
  return off < wa || off + wb > s;
}

// Checks and parameters shared by the two directions. `none`: weights absent (no norm).
fa_status rope_setup(RopeParams& p, const void* q_weight, const void* k_weight, float eps, const int32_t* positions,
                     const float* inv_freq, int num_axes, const int32_t* sections, int rot_dim, int interleaved,
                     int64_t T, int Hq, int Hkv, int d) {
  if (T < 0 || Hq <= 0 || Hkv <= 0 || rot_dim < 0 || (q_weight == nullptr) != (k_weight == nullptr))
    return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (rot_dim > d || (rot_dim == 0 && !q_weight)) return FA_ERR_INVALID_ARG;
  if (q_weight && !(std::isfinite(eps) && eps > 0.f)) return FA_ERR_INVALID_ARG;
  if (rot_dim > 0) {
    if ((!positions && T > 0) || !inv_freq) return FA_ERR_INVALID_ARG;
    if (rot_dim % 16 != 0) return FA_ERR_UNSUPPORTED;
    if (num_axes < 1 || (num_axes > 1 && !sections)) return FA_ERR_INVALID_ARG;
    if (num_axes > kMaxAxes) return FA_ERR_UNSUPPORTED;
  }
  if (T > (1LL << 31) - 1 || (int64_t)Hq + Hkv > (1 << 20)) return FA_ERR_UNSUPPORTED;
  std::memset(&p, 0, sizeof(p));
  int end = 0;
  for (int a = 0; a < kMaxAxes - 1; ++a) p.section_end[a] = rot_dim / 2;
  if (rot_dim > 0 && sections) {
    for (int a = 0; a < num_axes; ++a) {
      if (sections[a] < 0 || sections[a] > rot_dim / 2) return FA_ERR_INVALID_ARG;
      end += sections[a];
      if (a < kMaxAxes - 1) p.section_end[a] = end;
    }
    if (end != rot_dim / 2) return FA_ERR_INVALID_ARG;
  }
  if (!is_aligned(q_weight, 16) || !is_aligned(k_weight, 16) || !is_aligned(positions, 4) || !is_aligned(inv_freq, 4))
    return FA_ERR_ALIGNMENT;
  p.w[0] = static_cast<const uint16_t*>(q_weight);
  p.w[1] = static_cast<const uint16_t*>(k_weight);
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.T = T;
  p.heads[0] = Hq;
  p.heads[1] = Hkv;
  const int per_pass = 32 / (d / 16);
  p.passes[0] = (Hq + per_pass - 1) / per_pass;
  p.passes[1] = (Hkv + per_pass - 1) / per_pass;
  p.rot = rot_dim;
  p.eps = eps;
  return FA_OK;
}

// A row tensor that must be present (unless there are no tokens).
fa_status check_rows(const Rows& r, int64_t T, int d) {
  if (T == 0) return FA_OK;
  if (!r.ptr || r.stride < (int64_t)r.heads * d) return FA_ERR_INVALID_ARG;
  if (r.stride > (1LL << 40) / T) return FA_ERR_UNSUPPORTED;
  if (!is_aligned(r.ptr, 16) || r.stride % 8 != 0) return FA_ERR_ALIGNMENT;
  return FA_OK;
}

// An output may be one of the inputs itself (same pointer and stride: each element is read before it
// is written, by the same thread); otherwise the two share nothing.
bool bad_output(const Rows& out, const Rows& in, int64_t T, int d) {
  if (out.ptr == in.ptr && out.stride == in.stride && out.heads == in.heads) return false;
  return rows_overlap(out, in, T, d);
}

}  // namespace
}  // namespace fa

extern "C" fa_status fa_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                     const void* q_weight, const void* k_weight, float eps, const int32_t* positions,
                                     const float* inv_freq, int num_axes, const int32_t* sections, int rot_dim,
                                     int interleaved, int64_t T, int Hq, int Hkv, int d, void* q_out,
                                     int64_t q_out_stride, void* k_out, int64_t k_out_stride, fa_stream_t stream) {
  fa::RopeParams p;
  fa_status err = fa::rope_setup(p, q_weight, k_weight, eps, positions, inv_freq, num_axes, sections, rot_dim,
                                 interleaved, T, Hq, Hkv, d);
  if (err != FA_OK) return err;
  const fa::Rows in[2] = {{q, q_stride, Hq}, {k, k_stride, Hkv}};
  const fa::Rows out[2] = {{q_out, q_out_stride, Hq}, {k_out, k_out_stride, Hkv}};
  for (int x = 0; x < 2; ++x) {
    if ((err = fa::check_rows(in[x], T, d)) != FA_OK || (err = fa::check_rows(out[x], T, d)) != FA_OK) return err;
    if (fa::bad_output(out[x], in[x], T, d) || fa::rows_overlap(out[x], in[1 - x], T, d)) return FA_ERR_INVALID_ARG;
    p.x[x] = static_cast<const uint16_t*>(in[x].ptr);
    p.x_stride[x] = in[x].stride;
    p.out[x] = static_cast<uint16_t*>(const_cast<void*>(out[x].ptr));
    p.out_stride[x] = out[x].stride;
  }
  if (fa::rows_overlap(out[0], out[1], T, d)) return FA_ERR_INVALID_ARG;
  fa::DeviceStatus* status = nullptr;
  int sm_count = 0;
  const int rc = fa::current_device_info(&status, &sm_count);
  if (rc != FA_OK) return (fa_status)rc;
  if (T == 0) return FA_OK;
  const fa::RopeSplit s = fa::split_rope(T, p.passes[0] + p.passes[1], sm_count);
  p.parts = s.parts;
  p.per_part = s.per_part;
  const bool norm = q_weight != nullptr;
  const cudaError_t e = d == 128 ? fa::launch_rope<128, false>(p, s.blocks, norm, interleaved != 0, stream)
                                 : fa::launch_rope<64, false>(p, s.blocks, norm, interleaved != 0, stream);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

extern "C" size_t fa_qk_norm_rope_bwd_workspace_bytes(int64_t T, int Hq, int Hkv, int d) {
  if (T < 0 || Hq <= 0 || Hkv <= 0 || (d != 64 && d != 128)) return 0;
  fa::DeviceStatus* status = nullptr;
  int sm_count = 152;  // without a device the size is that of a full part
  fa::current_device_info(&status, &sm_count);
  if (sm_count <= 0) sm_count = 152;
  const int per_pass = 32 / (d / 16);
  const int64_t passes = ((int64_t)Hq + per_pass - 1) / per_pass + ((int64_t)Hkv + per_pass - 1) / per_pass;
  if (passes > (1 << 20)) return 0;
  return (size_t)fa::split_rope(T, (int)passes, sm_count).blocks * 2 * d * sizeof(float);
}

extern "C" fa_status fa_qk_norm_rope_bwd(const void* dq_out, int64_t dq_out_stride, const void* dk_out,
                                         int64_t dk_out_stride, const void* q, int64_t q_stride, const void* k,
                                         int64_t k_stride, const void* q_weight, const void* k_weight, float eps,
                                         const int32_t* positions, const float* inv_freq, int num_axes,
                                         const int32_t* sections, int rot_dim, int interleaved, int64_t T, int Hq,
                                         int Hkv, int d, void* dq, int64_t dq_stride, void* dk, int64_t dk_stride,
                                         float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                                         fa_stream_t stream) {
  fa::RopeParams p;
  fa_status err = fa::rope_setup(p, q_weight, k_weight, eps, positions, inv_freq, num_axes, sections, rot_dim,
                                 interleaved, T, Hq, Hkv, d);
  if (err != FA_OK) return err;
  const bool norm = q_weight != nullptr;
  if (norm && (!dq_weight || !dk_weight)) return FA_ERR_INVALID_ARG;
  const fa::Rows grad[2] = {{dq_out, dq_out_stride, Hq}, {dk_out, dk_out_stride, Hkv}};
  const fa::Rows in[2] = {{norm ? q : nullptr, q_stride, Hq}, {norm ? k : nullptr, k_stride, Hkv}};
  const fa::Rows out[2] = {{dq, dq_stride, Hq}, {dk, dk_stride, Hkv}};
  for (int x = 0; x < 2; ++x) {
    if ((err = fa::check_rows(grad[x], T, d)) != FA_OK || (err = fa::check_rows(out[x], T, d)) != FA_OK) return err;
    if (norm && (err = fa::check_rows(in[x], T, d)) != FA_OK) return err;
    if (fa::bad_output(out[x], grad[x], T, d) || fa::rows_overlap(out[x], grad[1 - x], T, d) ||
        fa::bad_output(out[x], in[x], T, d) || fa::rows_overlap(out[x], in[1 - x], T, d))
      return FA_ERR_INVALID_ARG;
    p.x[x] = static_cast<const uint16_t*>(in[x].ptr);
    p.x_stride[x] = in[x].stride;
    p.dy[x] = static_cast<const uint16_t*>(grad[x].ptr);
    p.dy_stride[x] = grad[x].stride;
    p.out[x] = static_cast<uint16_t*>(const_cast<void*>(out[x].ptr));
    p.out_stride[x] = out[x].stride;
  }
  if (fa::rows_overlap(out[0], out[1], T, d)) return FA_ERR_INVALID_ARG;
  if (!fa::is_aligned(dq_weight, 4) || !fa::is_aligned(dk_weight, 4)) return FA_ERR_ALIGNMENT;
  fa::DeviceStatus* status = nullptr;
  int sm_count = 0;
  const int rc = fa::current_device_info(&status, &sm_count);
  if (rc != FA_OK) return (fa_status)rc;
  const fa::RopeSplit s = fa::split_rope(T, p.passes[0] + p.passes[1], sm_count);
  const size_t need = norm ? (size_t)s.blocks * 2 * d * sizeof(float) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need)) return FA_ERR_WORKSPACE;
  if (need > 0 && !fa::is_aligned(workspace, 256)) return FA_ERR_ALIGNMENT;
  p.parts = s.parts;
  p.per_part = s.per_part;
  p.partial = static_cast<float*>(workspace);
  if (T > 0) {
    const cudaError_t e = d == 128 ? fa::launch_rope<128, true>(p, s.blocks, norm, interleaved != 0, stream)
                                   : fa::launch_rope<64, true>(p, s.blocks, norm, interleaved != 0, stream);
    if (e != cudaSuccess) return FA_ERR_CUDA;
  }
  if (!norm) return FA_OK;
  fa::rope_weight_grad_kernel<<<2 * d / 32, 256, 0, stream>>>(p.partial, s.blocks, d, dq_weight, dk_weight);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
