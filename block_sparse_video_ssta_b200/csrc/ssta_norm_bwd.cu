// Backward of the norms around a block.  Per row, with rh = norm(r), yh = post_norm(y)
// (none: y) and g = dn * w * (1 + scale):
//   dR = dr + rstd * (g - mean(g) - rh * mean(g * rh)),   dx = res_scale * dR,
//   dh = dR * gate * pw,   dy = dh or prstd * (dh - mean(dh) - yh * mean(dh * yh)),
// and three sums per channel over the rows of each modulation group,
//   S1 = sum dn,  S2 = sum dn * rh,  S3 = sum dR * yh,
// from which every vector's gradient follows (dshift = S1, dscale = w S2, dgate = pw S3,
// dw = sum_g (1 + scale_g) S2_g, dpw = sum_g gate_g S3_g).
//
// A block walks a run of rows of one group, so a thread keeps the same eight channels
// throughout: its share of S1-S3 and the products of the vectors stay in registers, and
// the sums leave the SM once per run instead of once per row.  The rows ahead come by
// cp.async into slots of shared memory that only the copying thread reads: several rows
// are in flight per thread without registers and without a barrier.  r and y may be 8-bit
// checkpoints: their codes are what is copied, and they are decoded on the way to
// registers, which saves one of the two bytes of a bf16 read.  Two small kernels add the
// runs' sums in a fixed order (no atomics: equal inputs give equal bytes).
#include "ssta_norm.h"
#include "ssta_rows.cuh"

#include <algorithm>
#include <atomic>

namespace ssta {
namespace {

using namespace rows;

constexpr int kSms = 148;
constexpr int kSums = 3;   // S1, S2, S3
constexpr int kNeedS1 = 1, kNeedS2 = 2, kNeedS3 = 4;

struct BwdParams {
  NormBwdArgs a;
  float* partial;   // [groups * chunks][kSums][C]
  uint32_t rows, mod_rows, chunk_rows;
  int64_t mod_stride;
  int C, norm, post_norm, groups_per_row, format;
  int row_threads, slots, chunks, need;
  float inv_c, res_scale;
  bool param_f32;
};

// Threads of a row, rows at a time and runs per group; the same for every type, so that
// the workspace follows from the descriptor.
struct BwdShape {
  int row_threads, slots, chunks;
  uint32_t chunk_rows;
};

BwdShape bwd_shape(const NormGeom& g) {
  BwdShape b{};
  if (g.C <= 128) {
    b.row_threads = 16;
    b.slots = 16;
  } else {
    b.row_threads = (g.C / kVec + 31) / 32 * 32;
    b.slots = std::max(1, 256 / b.row_threads);
  }
  // Runs per group: as many blocks as the SMs hold at once (or a small multiple, whichever
  // leaves the fewest idle in the last wave), of at least four rows per slot.
  const int64_t resident = (int64_t)kSms * (b.row_threads * b.slots <= 256 ? 2 : 1);
  const int64_t most = std::max<int64_t>(1, (g.mod_rows + 4 * b.slots - 1) / (4 * b.slots));
  int64_t chunks = 1;
  double best = 0;
  for (int64_t waves = 1; waves <= 4; ++waves) {
    const int64_t c = std::min(most, std::max<int64_t>(1, resident * waves / g.groups));
    const int64_t blocks = c * g.groups, full = (blocks + resident - 1) / resident * resident;
    if ((double)blocks / full > best + 0.02) {
      best = (double)blocks / full;
      chunks = c;
    }
  }
  const int64_t per = (g.mod_rows + chunks - 1) / chunks;
  b.chunk_rows = (uint32_t)((per + b.slots - 1) / b.slots * b.slots);
  b.chunks = (int)((g.mod_rows + b.chunk_rows - 1) / b.chunk_rows);
  return b;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A thread's slot for one vector of a dense tensor: 16-byte planes, one entry per thread
// in each (neighbouring threads' 16 bytes are neighbours, no bank conflicts).
template <typename T> constexpr int kPlanes = (int)sizeof(T) * kVec / 16;
template <typename T> __device__ __forceinline__ void copy_dense(uint32_t slot, int threads, const T* src) {
#pragma unroll
  for (int i = 0; i < kPlanes<T>; ++i) cp_async16(slot + (i * threads + threadIdx.x) * 16, reinterpret_cast<const char*>(src) + 16 * i);
}
__device__ __forceinline__ Raw<__nv_bfloat16> read_dense(const uint8_t* slot, int, __nv_bfloat16) {
  return {reinterpret_cast<const uint4*>(slot)[threadIdx.x]};
}
__device__ __forceinline__ Raw<float> read_dense(const uint8_t* slot, int threads, float) {
  return {reinterpret_cast<const float4*>(slot)[threadIdx.x], reinterpret_cast<const float4*>(slot)[threads + threadIdx.x]};
}

// The sums of a and b over the threads of a row.  HALF: a row is half a warp.
template <bool HALF>
__device__ __forceinline__ void row_sum2(float& a, float& b, const BwdParams& p, float2* exchange, int slot) {
#pragma unroll
  for (int off = HALF ? 8 : 16; off > 0; off >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, off);
    b += __shfl_xor_sync(0xffffffffu, b, off);
  }
  if constexpr (!HALF) {
    const int warps = p.row_threads >> 5;
    if (warps > 1) {
      if ((threadIdx.x & 31) == 0) exchange[threadIdx.x >> 5] = make_float2(a, b);
      asm volatile("bar.sync %0, %1;" ::"r"(slot + 1), "r"(p.row_threads) : "memory");
      a = b = 0.f;
      for (int w = 0; w < warps; ++w) {
        const float2 e = exchange[slot * warps + w];
        a += e.x;
        b += e.y;
      }
    }
  }
}

template <typename T, bool CODES, bool POST, bool HALF, int MAXT>
struct Kernel {
  // bytes of a thread's slots per row: dn, dr, r and (behind a gated residual) y
  static constexpr int kDense = (int)sizeof(T) * kVec, kKept = CODES ? 8 : kDense;
  static constexpr int kRowBytes = 2 * kDense + (POST ? 2 : 1) * kKept;
  // rows in flight: four where two blocks still share an SM, fewer for the widest rows
  static constexpr int kFit = (MAXT <= 256 ? 110 : 200) * 1024 / (MAXT * kRowBytes);
  static constexpr int kStages = kFit < 1 ? 1 : kFit < 4 ? kFit : 4;
  static constexpr int kSmem = (kStages * kRowBytes > kSums * kVec * 4 ? kStages * kRowBytes : kSums * kVec * 4) * MAXT;
};

template <typename T, bool CODES, bool POST, bool HALF, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT <= 256 ? 2 : 1) norm_bwd_kernel(const __grid_constant__ BwdParams p) {
  using K = Kernel<T, CODES, POST, HALF, MAXT>;
  extern __shared__ __align__(16) uint8_t stage[];
  __shared__ float2 exchange[2][2][MAXT / 32];
  const NormBwdArgs& a = p.a;
  const int threads = blockDim.x;
  const int slot = HALF ? threadIdx.x >> 4 : threadIdx.x / p.row_threads;
  const int lane = HALF ? threadIdx.x & 15 : threadIdx.x % p.row_threads;
  const int ch = lane * kVec;
  const bool in = ch < p.C;
  const uint32_t item = blockIdx.x, grp = item / p.chunks, chunk = item % p.chunks;
  const int64_t first = (int64_t)grp * p.mod_rows + (int64_t)chunk * p.chunk_rows;
  const int64_t group_end = min((int64_t)(grp + 1) * p.mod_rows, (int64_t)p.rows);
  const int64_t last = min(first + p.chunk_rows, group_end);
  const int iters = last > first ? (int)((last - first + p.slots - 1) / p.slots) : 0;
  const bool has_n = a.dn != nullptr, has_r = a.dr != nullptr;
  const bool has_y = POST && (a.y != nullptr || a.y_saved.codes != nullptr);

  const uint32_t stage0 = (uint32_t)__cvta_generic_to_shared(stage);
  auto prefetch = [&](int it) {
    const int64_t row = first + (int64_t)it * p.slots + slot;
    if (in && it < iters && row < last) {
      const int64_t at = row * p.C + ch;
      uint32_t s = stage0 + (it % K::kStages) * K::kRowBytes * threads;
      if (has_n) copy_dense(s, threads, static_cast<const T*>(a.dn) + at);
      s += K::kDense * threads;
      if (has_r) copy_dense(s, threads, static_cast<const T*>(a.dr) + at);
      s += K::kDense * threads;
      if (has_n) {
        if constexpr (CODES) cp_async8(s + threadIdx.x * 8, static_cast<const uint8_t*>(a.r_saved.codes) + at);
        else copy_dense(s, threads, static_cast<const T*>(a.r) + at);
      }
      if constexpr (POST) {
        s += K::kKept * threads;
        if (has_y) {
          if constexpr (CODES) cp_async8(s + threadIdx.x * 8, static_cast<const uint8_t*>(a.y_saved.codes) + at);
          else copy_dense(s, threads, static_cast<const T*>(a.y) + at);
        }
      }
    }
    cp_commit();
  };
  // a row's scalars, fetched one row ahead into registers
  struct Scalars { float mean, rstd, pmean, prstd; int er, ey; };
  auto scalars = [&](int it) {
    Scalars v{0.f, 0.f, 0.f, 1.f, 1, 1};
    const int64_t row = first + (int64_t)it * p.slots + slot;
    if (in && it < iters && row < last) {
      if (has_n) {
        v.rstd = a.rstd[row];
        if (p.norm == SSTA_NORM_LAYER) v.mean = a.mean[row];
        if constexpr (CODES) v.er = a.r_saved.exponents[row * p.groups_per_row + ch / kGroup];
      }
      if constexpr (POST) {
        if (p.post_norm != SSTA_NORM_NONE) v.prstd = a.post_rstd[row];
        if (p.post_norm == SSTA_NORM_LAYER) v.pmean = a.post_mean[row];
        if constexpr (CODES) {
          if (has_y) v.ey = a.y_saved.exponents[row * p.groups_per_row + ch / kGroup];
        }
      }
    }
    return v;
  };

#pragma unroll
  for (int i = 0; i < K::kStages; ++i) prefetch(i);
  Scalars next = scalars(0);

  // products of the vectors for this thread's channels
  float gw[kVec], gp[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) gw[j] = gp[j] = 1.f;
  if (in) {
    const int64_t mod = (int64_t)grp * p.mod_stride + ch;
    float w[kVec];
    if (a.weight != nullptr) {
      load_param8(a.weight, ch, p.param_f32, w);
#pragma unroll
      for (int j = 0; j < kVec; ++j) gw[j] = w[j];
    }
    if (a.scale != nullptr) {
      load_param8(a.scale, mod, p.param_f32, w);
#pragma unroll
      for (int j = 0; j < kVec; ++j) gw[j] *= 1.f + w[j];
    }
    if constexpr (POST) {
      if (a.post_weight != nullptr) {
        load_param8(a.post_weight, ch, p.param_f32, w);
#pragma unroll
        for (int j = 0; j < kVec; ++j) gp[j] = w[j];
      }
      if (a.gate != nullptr) {
        load_param8(a.gate, mod, p.param_f32, w);
#pragma unroll
        for (int j = 0; j < kVec; ++j) gp[j] *= w[j];
      }
    }
  }
  float s1[kVec], s2[kVec], s3[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) s1[j] = s2[j] = s3[j] = 0.f;

  for (int it = 0; it < iters; ++it) {
    const Scalars sc = next;
    next = scalars(it + 1);
    cp_wait<K::kStages - 1>();
    const int64_t row = first + (int64_t)it * p.slots + slot;
    const bool alive = in && row < last;   // others carry zeros through the sums
    const uint8_t* s = stage + (it % K::kStages) * K::kRowBytes * threads;
    float dR[kVec], yh[POST ? kVec : 1];
#pragma unroll
    for (int j = 0; j < kVec; ++j) dR[j] = 0.f;
    if (has_r && alive) unpack(read_dense(s + K::kDense * threads, threads, T()), dR);
    if (has_n) {
      float dn[kVec], rh[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) dn[j] = rh[j] = 0.f;
      if (alive) {
        unpack(read_dense(s, threads, T()), dn);
        const uint8_t* sr = s + 2 * K::kDense * threads;
        if constexpr (CODES) decode8(reinterpret_cast<const uint2*>(sr)[threadIdx.x], sc.er, p.format, rh);
        else unpack(read_dense(sr, threads, T()), rh);
#pragma unroll
        for (int j = 0; j < kVec; ++j) rh[j] = (rh[j] - sc.mean) * sc.rstd;
      }
      float m1 = 0.f, m2 = 0.f;
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        s1[j] += dn[j];
        s2[j] = fmaf(dn[j], rh[j], s2[j]);
        dn[j] *= gw[j];
        m1 += dn[j];
        m2 = fmaf(dn[j], rh[j], m2);
      }
      row_sum2<HALF>(m1, m2, p, exchange[it & 1][0], slot);
      m1 = p.norm == SSTA_NORM_LAYER ? m1 * p.inv_c : 0.f;
      m2 *= p.inv_c;
#pragma unroll
      for (int j = 0; j < kVec; ++j) dR[j] = fmaf(sc.rstd, dn[j] - m1 - rh[j] * m2, dR[j]);
    }
    if (alive) {
      float out[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) out[j] = POST ? p.res_scale * dR[j] : dR[j];
      store8(static_cast<T*>(a.dx) + row * p.C + ch, out);
    }
    if constexpr (POST) {
      if (has_y) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) yh[j] = 0.f;
        if (alive) {
          const uint8_t* sy = s + (2 * K::kDense + K::kKept) * threads;
          if constexpr (CODES) decode8(reinterpret_cast<const uint2*>(sy)[threadIdx.x], sc.ey, p.format, yh);
          else unpack(read_dense(sy, threads, T()), yh);
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          if (p.post_norm != SSTA_NORM_NONE) yh[j] = alive ? (yh[j] - sc.pmean) * sc.prstd : 0.f;
          s3[j] = fmaf(dR[j], yh[j], s3[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < kVec; ++j) dR[j] *= gp[j];
      if (p.post_norm != SSTA_NORM_NONE) {
        float m1 = 0.f, m2 = 0.f;
        if (alive) {   // dR holds the norm's row terms also where no channel is
#pragma unroll
          for (int j = 0; j < kVec; ++j) {
            m1 += dR[j];
            m2 = fmaf(dR[j], yh[j], m2);
          }
        }
        row_sum2<HALF>(m1, m2, p, exchange[it & 1][1], slot);
        m1 = p.post_norm == SSTA_NORM_LAYER ? m1 * p.inv_c : 0.f;
        m2 *= p.inv_c;
#pragma unroll
        for (int j = 0; j < kVec; ++j) dR[j] = sc.prstd * (dR[j] - m1 - yh[j] * m2);
      }
      if (alive) store8(static_cast<T*>(a.dy) + row * p.C + ch, dR);
    }
    prefetch(it + K::kStages);   // into the slot just read
  }

  if (p.need == 0) return;
  cp_wait<0>();
  if (p.slots > 1) {
    // slot 0 adds the other slots' sums in order; the staging memory is free now
    __syncthreads();
    float* f = reinterpret_cast<float*>(stage);
    const int rt = HALF ? 16 : p.row_threads;
    auto at = [&](int s, int j) -> float& { return f[(s * kSums * kVec + j) * rt + lane]; };
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      at(slot, j) = s1[j];
      at(slot, kVec + j) = s2[j];
      at(slot, 2 * kVec + j) = s3[j];
    }
    __syncthreads();
    if (slot > 0) return;
    for (int o = 1; o < p.slots; ++o) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        s1[j] += at(o, j);
        s2[j] += at(o, kVec + j);
        s3[j] += at(o, 2 * kVec + j);
      }
    }
  }
  if (!in) return;
  float* out = p.partial + (int64_t)item * kSums * p.C + ch;
  if (p.need & kNeedS1) store8(out, s1);
  if (p.need & kNeedS2) store8(out + p.C, s2);
  if (p.need & kNeedS3) store8(out + 2 * (int64_t)p.C, s3);
}

// Sums of the runs of each group, in order, and the modulation's gradients from them;
// leaves the group's term of dweight and dpost_weight in its first run's place (or, with
// one group, writes the gradient).  32 channels per block; 8 threads per channel share a
// group's runs, or take a group each where a group has few runs.
constexpr int kFinalY = 8;
struct FinalParams {
  BwdParams b;
  uint32_t groups;
  int channel_blocks;
  bool per_group;   // a group per thread row
};

__global__ void __launch_bounds__(32 * kFinalY) norm_bwd_groups_kernel(const __grid_constant__ FinalParams f) {
  const BwdParams& p = f.b;
  const NormBwdArgs& a = p.a;
  __shared__ float part[kSums][kFinalY][32];
  const int c = (blockIdx.x % f.channel_blocks) * 32 + threadIdx.x;
  const uint32_t gb = blockIdx.x / f.channel_blocks;
  const int64_t grp = f.per_group ? (int64_t)gb * kFinalY + threadIdx.y : gb;
  const bool in = c < p.C && grp < f.groups;
  const int start = f.per_group ? 0 : threadIdx.y, step = f.per_group ? 1 : kFinalY;
  float s[kSums] = {0.f, 0.f, 0.f};
  float* base = p.partial + grp * p.chunks * kSums * p.C + c;
  if (in) {
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
      if (!(p.need & (1 << k))) continue;
      const float* q = base + (int64_t)k * p.C;
#pragma unroll 8
      for (int i = start; i < p.chunks; i += step) s[k] += q[(int64_t)i * kSums * p.C];
    }
  }
  if (!f.per_group) {
#pragma unroll
    for (int k = 0; k < kSums; ++k) part[k][threadIdx.y][threadIdx.x] = s[k];
    __syncthreads();
    if (threadIdx.y > 0) return;
#pragma unroll
    for (int k = 0; k < kSums; ++k)
      for (int y = 1; y < kFinalY; ++y) s[k] += part[k][y][threadIdx.x];
  }
  if (!in) return;
  auto param = [&](const void* v, int64_t i) {
    return p.param_f32 ? static_cast<const float*>(v)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(v)[i]);
  };
  const int64_t mod = grp * p.mod_stride + c, out = grp * p.C + c;
  if (a.dshift != nullptr) a.dshift[out] = s[0];
  if (a.dscale != nullptr) a.dscale[out] = a.weight != nullptr ? s[1] * param(a.weight, c) : s[1];
  if (a.dgate != nullptr) a.dgate[out] = a.post_weight != nullptr ? s[2] * param(a.post_weight, c) : s[2];
  if (a.dweight != nullptr) {
    const float t = a.scale != nullptr ? fmaf(s[1], param(a.scale, mod), s[1]) : s[1];
    if (f.groups == 1) a.dweight[c] = t; else base[p.C] = t;
  }
  if (a.dpost_weight != nullptr) {
    const float t = a.gate != nullptr ? s[2] * param(a.gate, mod) : s[2];
    if (f.groups == 1) a.dpost_weight[c] = t; else base[2 * (int64_t)p.C] = t;
  }
}

// dweight and dpost_weight: the groups' terms in order, 32 threads per channel.
__global__ void __launch_bounds__(1024) norm_bwd_weights_kernel(const __grid_constant__ FinalParams f) {
  const BwdParams& p = f.b;
  __shared__ float part[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float* const outs[2] = {p.a.dweight, p.a.dpost_weight};
  for (int k = 0; k < 2; ++k) {
    if (outs[k] == nullptr) continue;
    float s = 0.f;
    if (c < p.C) {
      const float* q = p.partial + (int64_t)(k + 1) * p.C + c;
#pragma unroll 2
      for (int64_t g = threadIdx.y; g < f.groups; g += 32) s += q[g * p.chunks * kSums * p.C];
    }
    __syncthreads();
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < p.C) {
      for (int y = 1; y < 32; ++y) s += part[y][threadIdx.x];
      outs[k][c] = s;
    }
  }
}

template <typename T, bool CODES, bool POST, bool HALF, int MAXT>
cudaError_t launch_rows(const BwdParams& p, unsigned blocks, int threads, cudaStream_t s) {
  using K = Kernel<T, CODES, POST, HALF, MAXT>;
  const int smem = K::kSmem / MAXT * threads;
  static std::atomic<bool> attr_set[64];
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kernel = norm_bwd_kernel<T, CODES, POST, HALF, MAXT>;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, K::kSmem);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  kernel<<<blocks, threads, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T, bool CODES, bool POST>
cudaError_t launch_shape(const BwdParams& p, unsigned blocks, cudaStream_t s) {
  const int threads = p.row_threads * p.slots;
  if (p.row_threads == 16) return launch_rows<T, CODES, POST, true, 256>(p, blocks, threads, s);
  if (threads <= 256) return launch_rows<T, CODES, POST, false, 256>(p, blocks, threads, s);
  if (threads <= 512) return launch_rows<T, CODES, POST, false, 512>(p, blocks, threads, s);
  return launch_rows<T, CODES, POST, false, 1024>(p, blocks, threads, s);
}

template <typename T>
cudaError_t launch_type(const BwdParams& p, unsigned blocks, cudaStream_t s) {
  const bool codes = p.a.r_saved.codes != nullptr || p.a.y_saved.codes != nullptr;
  if (p.a.dy != nullptr)
    return codes ? launch_shape<T, true, true>(p, blocks, s) : launch_shape<T, false, true>(p, blocks, s);
  return codes ? launch_shape<T, true, false>(p, blocks, s) : launch_shape<T, false, false>(p, blocks, s);
}

}  // namespace

size_t norm_bwd_workspace_bytes(const NormGeom& g) {
  const BwdShape b = bwd_shape(g);
  const size_t bytes = (size_t)g.groups * b.chunks * kSums * g.C * sizeof(float);
  return (bytes + 255) / 256 * 256;
}

cudaError_t launch_norm_bwd(const NormGeom& g, const NormBwdArgs& a, void* workspace, cudaStream_t s) {
  const BwdShape shape = bwd_shape(g);
  FinalParams f{};
  BwdParams& p = f.b;
  p.a = a;
  p.partial = static_cast<float*>(workspace);
  p.rows = (uint32_t)g.rows;
  p.mod_rows = (uint32_t)g.mod_rows;
  p.chunk_rows = shape.chunk_rows;
  p.mod_stride = g.mod_stride;
  p.C = g.C;
  p.norm = g.norm;
  p.post_norm = g.post_norm;
  p.groups_per_row = groups_per_row(g.C);
  p.format = a.r_saved.codes != nullptr ? a.r_saved.format : a.y_saved.format;
  p.row_threads = shape.row_threads;
  p.slots = shape.slots;
  p.chunks = shape.chunks;
  p.need = (a.dshift != nullptr ? kNeedS1 : 0) | (a.dscale != nullptr || a.dweight != nullptr ? kNeedS2 : 0) |
           (a.dgate != nullptr || a.dpost_weight != nullptr ? kNeedS3 : 0);
  p.inv_c = 1.0f / (float)g.C;
  p.res_scale = g.res_scale;
  p.param_f32 = g.param_f32;
  f.groups = (uint32_t)g.groups;
  f.channel_blocks = (g.C + 31) / 32;
  f.per_group = shape.chunks < kFinalY && g.groups > 1;
  const int64_t items = g.groups * shape.chunks;
  const int64_t group_blocks = (f.per_group ? (g.groups + kFinalY - 1) / kFinalY : g.groups) * f.channel_blocks;
  if (items > INT32_MAX || group_blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaError_t e = g.bf16 ? launch_type<__nv_bfloat16>(p, (unsigned)items, s) : launch_type<float>(p, (unsigned)items, s);
  if (e != cudaSuccess || p.need == 0) return e;
  norm_bwd_groups_kernel<<<(unsigned)group_blocks, dim3(32, kFinalY), 0, s>>>(f);
  if (g.groups > 1 && (a.dweight != nullptr || a.dpost_weight != nullptr))
    norm_bwd_weights_kernel<<<(g.C + 31) / 32, dim3(32, 32), 0, s>>>(f);
  return cudaGetLastError();
}

}  // namespace ssta
