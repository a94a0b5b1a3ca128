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
// cp.async into slots of shared memory that only the copying thread (fp32: its warp)
// reads: several rows are in flight per thread without registers and without a block-wide
// barrier (channels and rows that do not exist are filled with zeros there, so the
// arithmetic has no conditions).
// r and y may be 8-bit checkpoints: their codes are what is copied, and they are decoded
// on the way to registers, which saves one of the two bytes of a bf16 read.  A small
// kernel adds the runs' sums in a fixed order (no atomics: equal inputs give equal bytes).
//
// What bounds it: HBM, once the instructions fit.  A thread handles two rows at a time and
// works on pairs of channels; the row sums of both rows share one butterfly, in which a
// lane gives away the sums that it need not finish (6 shuffles for four sums instead of
// 20).  219,600 x 2,048 bf16 (gradients of r and n in, of x and y out), passes back to back:
// 754-813 us from int8 checkpoints, 0.85-0.91 of the measured copy rate (the power cap decides
// which; 725 us, 0.95, with L2 flushed between passes), 967 us dense, 0.85 (910 us, 0.90).
// One row at a time in scalar arithmetic took 1,165 and 986 us with pauses.  Rows of 128
// channels (heads): 1,785,600 of them take 262 us from dense rows (0.80) and from int8 (0.67)
// alike, so what bounds them is not the bytes.  A modulation row per token makes every run one
// row: 6.1 ms dense for 219,600 x 2,048 (0.32, fp32 gradients of the modulation included), and
// the runs' sums take 5.4 GB.
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
  // what is copied row by row; an absent tensor has some valid address and reads as zeros
  const void *dn, *dr, *r, *y;
  bool has_n, has_r, has_y;
  float* partial;   // [groups * chunks][kSums][C]
  uint32_t rows, mod_rows, chunk_rows;
  int64_t mod_stride;
  int C, norm, post_norm, groups_per_row, format;
  int row_threads, slots, chunks, need;
  float inv_c, res_scale;
  bool param_f32;
};

// Threads of a row, rows at once (slots; each takes U at a time) and runs per group; the
// same for every type, so that the workspace follows from the descriptor.
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
    const int vecs = g.C <= 4096 ? g.C / kVec : (g.C / kVec + 1) / 2;   // above, two vectors per thread
    b.row_threads = (vecs + 31) / 32 * 32;
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

// Copies to shared memory; zeros instead where `live` is false (the address is not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(live ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// One vector of a dense tensor per thread of the block in shared memory.  fp32: the LANES
// lanes of a row's part copy it in order, 16 bytes per lane and step, so a thread copies
// partly for others and warps synchronise around it.  (Each thread copying its own 32 bytes
// fetches every sector twice, and splitting the halves into two planes for conflict-free
// reads makes the copies scatter: 334 us instead of 213 us for 49,290 x 1,544.)
template <typename T, int MAXT> constexpr int kDenseBytes = (int)sizeof(T) * kVec * MAXT;

// `off` is the offset of channel `ch`, the thread's first, from src; src itself is always
// valid to address.
template <int MAXT, int LANES>
__device__ __forceinline__ void copy_dense(uint32_t slot, const __nv_bfloat16* src, uint32_t off, int ch, int C, bool live) {
  const bool ok = live && ch < C;
  cp_async16(slot + threadIdx.x * 16, src + (ok ? off : 0), ok);
}
template <int MAXT, int LANES>
__device__ __forceinline__ void copy_dense(uint32_t slot, const float* src, uint32_t off, int ch, int C, bool live) {
  const int l = threadIdx.x % LANES;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int c = l + j * LANES;                 // 16-byte chunk among those of LANES vectors
    const int d = c * 4 - l * kVec;              // from this thread's own first channel
    const bool ok = live && ch + d < C;
    cp_async16(slot + (threadIdx.x - l) * 32 + c * 16, src + (ok ? off + d : 0), ok);
  }
}
template <int MAXT>
__device__ __forceinline__ V8 read_dense(const uint8_t* slot, __nv_bfloat16) {
  return unpack(Raw<__nv_bfloat16>{reinterpret_cast<const uint4*>(slot)[threadIdx.x]});
}
template <int MAXT>
__device__ __forceinline__ V8 read_dense(const uint8_t* slot, float) {
  return unpack(Raw<float>{reinterpret_cast<const float4*>(slot)[2 * threadIdx.x],
                           reinterpret_cast<const float4*>(slot)[2 * threadIdx.x + 1]});
}

// Sums of a[u] and b[u] over the threads of each of U rows (1 or 2); every thread of the
// rows gets them.  A row is a half-warp (HALF) or `warps` warps.  In the first steps a lane
// keeps half of its sums and hands the others to its partner, so each sum ends in a part
// of the lanes, from which the warps' parts are added and handed round.
template <bool HALF, int U>
__device__ __forceinline__ void row_sums(float (&a)[U], float (&b)[U], int warps, float* exchange, int slot) {
  constexpr unsigned kAll = 0xffffffffu;
  constexpr int kLanes = HALF ? 16 : 32;
  const int lane = threadIdx.x & 31;
  int off = kLanes / 2;
  float x, y;
  if constexpr (U == 2) {
    const bool up = lane & off;
    x = (up ? a[1] : a[0]) + __shfl_xor_sync(kAll, up ? a[0] : a[1], off);
    y = (up ? b[1] : b[0]) + __shfl_xor_sync(kAll, up ? b[0] : b[1], off);
    off /= 2;
  } else {
    x = a[0];
    y = b[0];
  }
  const bool up = lane & off;
  float v = (up ? y : x) + __shfl_xor_sync(kAll, up ? x : y, off);
  const int part = off;   // lanes holding one sum: its index is the lane over `part`
#pragma unroll
  for (off /= 2; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  const int first = lane & ~(kLanes - 1);
  if constexpr (!HALF) {
    if (warps > 1) {
      float* row = exchange + slot * warps * (2 * U);
      if (lane % part == 0) row[(lane / part) * warps + ((threadIdx.x >> 5) - slot * warps)] = v;
      asm volatile("bar.sync %0, %1;" ::"r"(slot + 1), "r"(warps * 32) : "memory");
      v = 0.f;
      for (int w = lane % part; w < warps; w += part) v += row[(lane / part) * warps + w];
#pragma unroll
      for (int o = part / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    a[u] = __shfl_sync(kAll, v, first + 2 * u * part);
    b[u] = __shfl_sync(kAll, v, first + (2 * u + 1) * part);
  }
}

// What a row brings besides its channels, in shared memory for kWindow rows at a time:
// xh = v * rstd + shift of both norms, and the codes' scales of each group.
constexpr int kWindow = 64;   // a multiple of the rows a block takes at once (at most 32)
struct RowScalars {
  float rstd, shift, prstd, pshift;
};

// What stands behind the norm's gradient: nothing, a gate, a gate and a post norm.
enum Post { kNoPost = 0, kGate = 1, kPostNorm = 2 };

// SRC: 0 dense r and y, 1 + format: checkpoints.
template <typename T, int SRC, int POST, bool HALF, int NV, int U, int MAXT>
struct Kernel {
  static constexpr int kKept = SRC ? 8 * MAXT : kDenseBytes<T, MAXT>;   // r, y
  // places of a vector's dn, dr, r and y
  static constexpr int kR = 2 * kDenseBytes<T, MAXT>, kY = kR + kKept, kVecBytes = POST ? kY + kKept : kY;
  static constexpr int kStageBytes = NV * U * kVecBytes;
  static constexpr int kScales = SRC ? MAXT * NV * kVec / kGroup : 0;   // group scales of a row
  static constexpr int kTable = kWindow * ((int)sizeof(RowScalars) + (POST ? 2 : 1) * kScales * 4);
  // With two vectors per thread and a gated residual the products of the parameter vectors do
  // not fit in registers beside the sums: each thread keeps its own in shared memory (100 M
  // bf16 elements in rows of 8,192 channels: 208 us instead of 255 us with the spills).  Dense
  // fp32 rows need that memory for copies in flight.
  static constexpr bool kShared = NV > 1 && POST && !(sizeof(T) == 4 && SRC == 0);
  static constexpr int kVectors = kShared ? NV * 2 * kVec * 4 * MAXT : 0;
  // copies in flight: up to four times U rows, as far as shared memory goes (two blocks of
  // 256 threads, or one larger one, per SM)
  static constexpr int kFit = ((MAXT <= 256 ? 112 : 224) * 1024 - kTable - kVectors) / kStageBytes;
  static constexpr int kStages = kFit < 1 ? 1 : kFit < 4 ? kFit : 4;
  static constexpr int kSumBytes = kSums * NV * kVec * 4 * MAXT;
  static constexpr int kSmem = kTable + kVectors + (kStages * kStageBytes > kSumBytes ? kStages * kStageBytes : kSumBytes);
};

template <typename T, int SRC, int POST, bool HALF, int NV, int U, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT <= 256 ? 2 : 1) norm_bwd_kernel(const __grid_constant__ BwdParams p) {
  using K = Kernel<T, SRC, POST, HALF, NV, U, MAXT>;
  constexpr int kLanes = HALF ? 16 : 32;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float exchange[2][2][2 * U * (MAXT / 32)];
  RowScalars* const table = reinterpret_cast<RowScalars*>(smem);
  float* const scales_r = reinterpret_cast<float*>(smem + kWindow * sizeof(RowScalars));
  float* const scales_y = scales_r + kWindow * K::kScales;
  float4* const vectors = reinterpret_cast<float4*>(smem + K::kTable);
  uint8_t* const stage = smem + K::kTable + K::kVectors;
  const NormBwdArgs& a = p.a;
  const int warps = p.row_threads >> 5;
  const int slot = HALF ? threadIdx.x >> 4 : threadIdx.x / p.row_threads;
  const int lane = HALF ? threadIdx.x & 15 : threadIdx.x % p.row_threads;
  const int step = p.row_threads * kVec;   // between a thread's vectors
  const uint32_t item = blockIdx.x, grp = item / p.chunks, chunk = item % p.chunks;
  const int64_t group_first = (int64_t)grp * p.mod_rows;
  const int64_t first = group_first + (int64_t)chunk * p.chunk_rows;
  const int64_t group_end = min(group_first + p.mod_rows, (int64_t)p.rows);
  const int count = (int)max(min((int64_t)p.chunk_rows, group_end - first), (int64_t)0);   // rows of this run
  const int per_iter = p.slots * U;
  bool in[NV];   // this vector's channels exist
#pragma unroll
  for (int i = 0; i < NV; ++i) in[i] = lane * kVec + i * step < p.C;
  // an element is addressed by the block's row (the same for all threads) and this offset
  const uint32_t mine = slot * U * p.C + lane * kVec;

  const uint32_t stage0 = (uint32_t)__cvta_generic_to_shared(stage);
  auto prefetch = [&](int done, int st) {   // rows done + slot * U .. into stage st
    const int64_t at = min(first + min(done, max(count - 1, 0)), (int64_t)p.rows - 1) * p.C;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool live = done + slot * U + u < count;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int ch = lane * kVec + i * step;
        const uint32_t off = mine + u * p.C + i * step, s = stage0 + st * K::kStageBytes + (u * NV + i) * K::kVecBytes;
        auto copy_kept = [&](uint32_t to, const void* src, bool has) {
          if constexpr (SRC) {
            const bool ok = live && has && in[i];
            cp_async8(to + threadIdx.x * 8, static_cast<const uint8_t*>(src) + at + (ok ? off : 0), ok);
          } else {
            copy_dense<MAXT, kLanes>(to, static_cast<const T*>(src) + at, off, ch, p.C, live && has);
          }
        };
        copy_dense<MAXT, kLanes>(s, static_cast<const T*>(p.dn) + at, off, ch, p.C, live && p.has_n);
        copy_dense<MAXT, kLanes>(s + kDenseBytes<T, MAXT>, static_cast<const T*>(p.dr) + at, off, ch, p.C, live && p.has_r);
        copy_kept(s + K::kR, p.r, p.has_n);
        if constexpr (POST) copy_kept(s + K::kY, p.y, p.has_y);
      }
    }
    cp_commit();
  };
  // Fills the table for the kWindow rows from w0 on (rstd and group scales 0 where there is
  // no row).  The first kWindow threads fetch the rows' scalars, the others the exponents.
  static_assert(kWindow < 160, "a block has at least 160 threads");
  auto fill_table = [&](int w0) {
    if (w0 > 0) __syncthreads();
    if (threadIdx.x < kWindow) {
      const int r = threadIdx.x;
      RowScalars v{0.f, 0.f, POST == kPostNorm ? 0.f : 1.f, 0.f};
      if (w0 + r < count) {
        const int64_t row = first + w0 + r;
        const bool layer = p.norm == SSTA_NORM_LAYER, post_layer = p.post_norm == SSTA_NORM_LAYER;
        const float rstd = p.has_n ? a.rstd[row] : 0.f, mean = p.has_n && layer ? a.mean[row] : 0.f;
        if constexpr (POST == kPostNorm) {
          const float prstd = a.post_rstd[row], pmean = post_layer ? a.post_mean[row] : 0.f;
          v.prstd = prstd;
          v.pshift = -pmean * prstd;
        }
        v.rstd = rstd;
        v.shift = -mean * rstd;
      }
      table[r] = v;
    } else if constexpr (SRC) {
      const int64_t from = (first + w0) * p.groups_per_row;
      const int n = min(kWindow, count - w0) * p.groups_per_row;
#pragma unroll 4
      for (int e = threadIdx.x - kWindow; e < kWindow * p.groups_per_row; e += blockDim.x - kWindow) {
        scales_r[e] = e < n && p.has_n ? code_scale(a.r_saved.exponents[from + e]) : 0.f;
        if constexpr (POST) scales_y[e] = e < n && p.has_y ? code_scale(a.y_saved.exponents[from + e]) : 0.f;
      }
    }
    __syncthreads();
  };

#pragma unroll
  for (int i = 0; i < K::kStages; ++i) prefetch(i * per_iter, i);

  // products of the vectors for this thread's channels (0 beyond C); all loads are issued
  // before the first is used
  V8 gw[NV], gp[POST ? NV : 1];
  auto products = [&](auto type) {
    using P = decltype(type);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = lane * kVec + i * step;
      const int64_t mod = (int64_t)grp * p.mod_stride + ch;
      Raw<P> w[4];
      const void* const src[4] = {a.weight, a.scale, a.post_weight, a.gate};
#pragma unroll
      for (int k = 0; k < (POST ? 4 : 2); ++k) {
        w[k] = zero_raw<P>();
        if (in[i] && src[k] != nullptr) w[k] = load_raw(static_cast<const P*>(src[k]) + (k & 1 ? mod : ch));
      }
      const float one = in[i] ? 1.f : 0.f;
      gw[i] = mul(a.weight != nullptr ? unpack(w[0]) : fill(one), add(unpack(w[1]), fill(one)));
      if constexpr (POST)
        gp[i] = mul(a.post_weight != nullptr ? unpack(w[2]) : fill(one), a.gate != nullptr ? unpack(w[3]) : fill(one));
    }
  };
  if (p.param_f32)
    products(float());
  else
    products(__nv_bfloat16());
  auto vector_place = [&](int k, int i) { return vectors + (k * NV + i) * 2 * MAXT + threadIdx.x; };
  if constexpr (K::kShared) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const Raw<float> r = pack(k ? gp[i] : gw[i], 0.f);
        vector_place(k, i)[0] = r.a;
        vector_place(k, i)[MAXT] = r.b;
      }
    }
  }
  auto product = [&](int k, int i) {   // 0: of the norm, 1: of the gate and the post norm
    if constexpr (K::kShared)
      return unpack(Raw<float>{vector_place(k, i)[0], vector_place(k, i)[MAXT]});
    else
      return k ? gp[POST ? i : 0] : gw[i];
  };
  V8 s1[NV], s2[NV], s3[POST ? NV : 1];
#pragma unroll
  for (int i = 0; i < NV; ++i) s1[i] = s2[i] = fill(0.f);
  if constexpr (POST) {
#pragma unroll
    for (int i = 0; i < NV; ++i) s3[i] = fill(0.f);
  }

  int st = 0, parity = 0;
  for (int done = 0; done < count; done += per_iter) {
    if (done % kWindow == 0) fill_table(done);
    cp_wait<K::kStages - 1>();
    if constexpr (sizeof(T) == 4) __syncwarp();
    const uint8_t* const s = stage + st * K::kStageBytes;
    const int wr = done % kWindow + slot * U;
    auto place = [&](int u, int i, int offset) { return s + (u * NV + i) * K::kVecBytes + offset; };
    // (value of r or y) * scale + shift, with the row's scale or the code group's
    auto kept = [&](int u, int i, int offset, const float* scales, float scale, float shift) {
      if constexpr (SRC) {
        scale *= scales[(wr + u) * p.groups_per_row + (in[i] ? (lane * kVec + i * step) / kGroup : 0)];
        return fma(decode8(reinterpret_cast<const uint2*>(place(u, i, offset))[threadIdx.x], SRC - 1), scale, shift);
      } else {
        return fma(read_dense<MAXT>(place(u, i, offset), T()), scale, shift);
      }
    };
    V8 g[U][NV], rh[U][NV];
    float m1[U], m2[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float2 rs = *reinterpret_cast<const float2*>(&table[wr + u].rstd);
      m1[u] = m2[u] = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const V8 dn = read_dense<MAXT>(place(u, i, 0), T());
        rh[u][i] = kept(u, i, K::kR, scales_r, rs.x, rs.y);
        s1[i] = add(s1[i], dn);
        s2[i] = fma(dn, rh[u][i], s2[i]);
        g[u][i] = mul(dn, product(0, i));
        m1[u] += sum(g[u][i]);
        m2[u] += dot(g[u][i], rh[u][i]);
      }
    }
    row_sums<HALF, U>(m1, m2, warps, exchange[parity][0], slot);
    T* const dx = static_cast<T*>(a.dx) + (first + done) * p.C;
    T* const dy = static_cast<T*>(a.dy) + (first + done) * p.C;
    V8 dR[U][NV], yh[POST ? U : 1][POST ? NV : 1];
    float q1[U], q2[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      q1[u] = q2[u] = 0.f;
      const RowScalars sc = table[wr + u];
      const float c1 = p.norm == SSTA_NORM_LAYER ? -sc.rstd * (m1[u] * p.inv_c) : 0.f;
      const float c2 = -sc.rstd * (m2[u] * p.inv_c);
      const bool live = done + slot * U + u < count;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t off = mine + u * p.C + i * step;
        dR[u][i] = add(read_dense<MAXT>(place(u, i, kDenseBytes<T, MAXT>), T()),
                       fma(sc.rstd, g[u][i], fma(rh[u][i], c2, c1)));
        if (live && in[i]) store8(dx + off, POST ? mul(dR[u][i], p.res_scale) : dR[u][i]);
        if constexpr (POST) {
          yh[u][i] = kept(u, i, K::kY, scales_y, sc.prstd, sc.pshift);
          s3[i] = fma(dR[u][i], yh[u][i], s3[i]);
          dR[u][i] = mul(dR[u][i], product(1, i));
          if constexpr (POST == kGate) {
            if (live && in[i]) store8(dy + off, dR[u][i]);
          } else {
            q1[u] += sum(dR[u][i]);
            q2[u] += dot(dR[u][i], yh[u][i]);
          }
        }
      }
    }
    if constexpr (POST == kPostNorm) {
      row_sums<HALF, U>(q1, q2, warps, exchange[parity][1], slot);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float prstd = table[wr + u].prstd;
        const float c1 = p.post_norm == SSTA_NORM_LAYER ? -prstd * (q1[u] * p.inv_c) : 0.f;
        const float c2 = -prstd * (q2[u] * p.inv_c);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (done + slot * U + u < count && in[i])
            store8(dy + (mine + u * p.C + i * step), fma(prstd, dR[u][i], fma(yh[u][i], c2, c1)));
        }
      }
    }
    // into the slots just read
    if constexpr (sizeof(T) == 4) __syncwarp();
    prefetch(done + K::kStages * per_iter, st);
    st = st + 1 == K::kStages ? 0 : st + 1;
    parity ^= 1;
  }

  // the next kernel's blocks may take the SMs that run out of rows (they wait for the sums)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (p.need == 0) return;
  cp_wait<0>();
  if constexpr (NV == 1) {
    if (p.slots > 1) {
      // slot 0 adds the other slots' sums in order; the staging memory is free now
      __syncthreads();
      uint64_t* f = reinterpret_cast<uint64_t*>(stage);
      const int rt = HALF ? 16 : p.row_threads;
      auto at = [&](int sl, int k, int j) -> uint64_t& { return f[((sl * kSums + k) * 4 + j) * rt + lane]; };
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        at(slot, 0, j) = s1[0].p[j];
        at(slot, 1, j) = s2[0].p[j];
        if constexpr (POST) at(slot, 2, j) = s3[0].p[j];
      }
      __syncthreads();
      if (slot > 0) return;
      for (int o = 1; o < p.slots; ++o) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s1[0].p[j] = f2_add(s1[0].p[j], at(o, 0, j));
          s2[0].p[j] = f2_add(s2[0].p[j], at(o, 1, j));
          if constexpr (POST) s3[0].p[j] = f2_add(s3[0].p[j], at(o, 2, j));
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (!in[i]) continue;
    float* out = p.partial + (int64_t)item * kSums * p.C + lane * kVec + i * step;
    if (p.need & kNeedS1) store8(out, s1[i]);
    if (p.need & kNeedS2) store8(out + p.C, s2[i]);
    if constexpr (POST) {
      if (p.need & kNeedS3) store8(out + 2 * (int64_t)p.C, s3[i]);
    }
  }
}

// The runs' sums, added in a fixed order, and every vector's gradient from them.  Launched
// as programmatic dependents of the kernel before: only their launch overlaps it.
struct FinalParams {
  BwdParams b;
  uint32_t groups;
  int channel_blocks;
  int slices;   // thread rows that share a group's runs
};

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Sum of every `step`th run from `start` of group `grp`, channel c.
__device__ __forceinline__ void sum_runs(const BwdParams& p, int64_t grp, int c, int start, int step, float (&s)[kSums]) {
  const volatile float* base = p.partial + grp * p.chunks * kSums * p.C + c;
#pragma unroll 4
  for (int i = start; i < p.chunks; i += step) {
    const volatile float* q = base + (int64_t)i * kSums * p.C;
#pragma unroll
    for (int k = 0; k < kSums; ++k) s[k] += p.need & (1 << k) ? q[(int64_t)k * p.C] : 0.f;
  }
}

// Writes the modulation's gradients of one group and channel from its sums; returns its
// terms of dweight and dpost_weight.
__device__ __forceinline__ float2 finish_group(const BwdParams& p, int64_t grp, int c, const float (&s)[kSums]) {
  const NormBwdArgs& a = p.a;
  auto param = [&](const void* v, int64_t i) {
    return p.param_f32 ? static_cast<const float*>(v)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(v)[i]);
  };
  const int64_t mod = grp * p.mod_stride + c, out = grp * p.C + c;
  if (a.dshift != nullptr) a.dshift[out] = s[0];
  if (a.dscale != nullptr) a.dscale[out] = a.weight != nullptr ? s[1] * param(a.weight, c) : s[1];
  if (a.dgate != nullptr) a.dgate[out] = a.post_weight != nullptr ? s[2] * param(a.post_weight, c) : s[2];
  float2 t = make_float2(0.f, 0.f);
  if (a.dweight != nullptr) t.x = a.scale != nullptr ? fmaf(s[1], param(a.scale, mod), s[1]) : s[1];
  if (a.dpost_weight != nullptr) t.y = a.gate != nullptr ? s[2] * param(a.gate, mod) : s[2];
  return t;
}

// Few groups (up to kFewGroups): one block does all groups of eight channels (one sector
// per run and sum), `slices` of its 64 thread rows sharing each group, so one launch
// finishes everything on as many SMs as there are sectors.
constexpr int kFewGroups = 64, kFinishX = 8, kFinishY = 64;
__global__ void __launch_bounds__(kFinishX * kFinishY) norm_bwd_finish_kernel(const __grid_constant__ FinalParams f) {
  const BwdParams& p = f.b;
  __shared__ float part[kSums][kFinishY][kFinishX];
  __shared__ float2 terms[kFinishY][kFinishX];
  const int x = threadIdx.x, y = threadIdx.y, c = blockIdx.x * kFinishX + x;   // C is a multiple of 8
  const int slice = y % f.slices, grp = y / f.slices;
  const bool mine = grp < f.groups;
  grid_dependency_wait();
  float s[kSums] = {0.f, 0.f, 0.f};
  if (mine) sum_runs(p, grp, c, slice, f.slices, s);
  // halve the slices of each group, then of all groups, in a fixed order
  for (int n = f.slices; n > 1;) {
    const int half = (n + 1) / 2;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSums; ++k) part[k][y][x] = s[k];
    __syncthreads();
    if (mine && slice + half < n) {
#pragma unroll
      for (int k = 0; k < kSums; ++k) s[k] += part[k][y + half][x];
    }
    n = half;
  }
  float2 t = make_float2(0.f, 0.f);
  if (mine && slice == 0) t = finish_group(p, grp, c, s);
  if (p.a.dweight == nullptr && p.a.dpost_weight == nullptr) return;
  if (slice == 0 && mine) terms[grp][x] = t;
  __syncthreads();
  if (y > 0) return;
  for (int o = 1; o < (int)f.groups; ++o) {
    t.x += terms[o][x].x;
    t.y += terms[o][x].y;
  }
  if (p.a.dweight != nullptr) p.a.dweight[c] = t.x;
  if (p.a.dpost_weight != nullptr) p.a.dpost_weight[c] = t.y;
}

// Many groups (of few runs each): a warp per group; the group's terms of dweight and
// dpost_weight take its first run's place, and a second kernel adds them.
constexpr int kGroupWarps = 8;
__global__ void __launch_bounds__(32 * kGroupWarps) norm_bwd_groups_kernel(const __grid_constant__ FinalParams f) {
  const BwdParams& p = f.b;
  const int c = (blockIdx.x % f.channel_blocks) * 32 + threadIdx.x;
  const int64_t grp = (int64_t)(blockIdx.x / f.channel_blocks) * kGroupWarps + threadIdx.y;
  grid_dependency_wait();
  if (c >= p.C || grp >= f.groups) return;
  float s[kSums] = {0.f, 0.f, 0.f};
  sum_runs(p, grp, c, 0, 1, s);
  const float2 t = finish_group(p, grp, c, s);
  float* base = p.partial + grp * p.chunks * kSums * p.C + c;
  if (p.a.dweight != nullptr) base[p.C] = t.x;
  if (p.a.dpost_weight != nullptr) base[2 * (int64_t)p.C] = t.y;
}

__global__ void __launch_bounds__(1024) norm_bwd_weights_kernel(const __grid_constant__ FinalParams f) {
  const BwdParams& p = f.b;
  __shared__ float part[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float* const outs[2] = {p.a.dweight, p.a.dpost_weight};
  grid_dependency_wait();
  for (int k = 0; k < 2; ++k) {
    if (outs[k] == nullptr) continue;
    float s = 0.f;
    if (c < p.C) {
      const volatile float* q = p.partial + (int64_t)(k + 1) * p.C + c;
#pragma unroll 4
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

// Launch as a programmatic dependent of the kernel before it on the stream.
cudaError_t launch_dependent(void (*kernel)(FinalParams), dim3 grid, dim3 block, const FinalParams& f, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, f);
}

template <typename T, int SRC, int POST, bool HALF, int NV, int U, int MAXT>
cudaError_t launch_rows(const BwdParams& p, unsigned blocks, int threads, cudaStream_t s) {
  using K = Kernel<T, SRC, POST, HALF, NV, U, MAXT>;
  static std::atomic<bool> attr_set[64];
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kernel = norm_bwd_kernel<T, SRC, POST, HALF, NV, U, MAXT>;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, K::kSmem);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  kernel<<<blocks, threads, K::kSmem, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int SRC, int POST>
cudaError_t launch_shape(const BwdParams& p, unsigned blocks, cudaStream_t s) {
  const int threads = p.row_threads * p.slots;
  constexpr int U = sizeof(T) == 4 && SRC == 0 && POST ? 1 : 2;   // four dense fp32 rows at once would fill the stage
  if (p.row_threads == 16) return launch_rows<T, SRC, POST, true, 1, U, 256>(p, blocks, threads, s);
  if (p.row_threads * kVec < p.C) return launch_rows<T, SRC, POST, false, 2, 1, 512>(p, blocks, threads, s);
  if (threads <= 256) return launch_rows<T, SRC, POST, false, 1, U, 256>(p, blocks, threads, s);
  return launch_rows<T, SRC, POST, false, 1, U, 512>(p, blocks, threads, s);
}

template <typename T, int POST>
cudaError_t launch_source(const BwdParams& p, unsigned blocks, cudaStream_t s) {
  if (p.a.r_saved.codes == nullptr && p.a.y_saved.codes == nullptr) return launch_shape<T, 0, POST>(p, blocks, s);
  return p.format == SSTA_INT8 ? launch_shape<T, 1 + SSTA_INT8, POST>(p, blocks, s)
                               : launch_shape<T, 1 + SSTA_E4M3, POST>(p, blocks, s);
}

template <typename T>
cudaError_t launch_type(const BwdParams& p, unsigned blocks, cudaStream_t s) {
  if (p.a.dy == nullptr) return launch_source<T, kNoPost>(p, blocks, s);
  return p.post_norm == SSTA_NORM_NONE ? launch_source<T, kGate>(p, blocks, s) : launch_source<T, kPostNorm>(p, blocks, s);
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
  p.has_n = a.dn != nullptr;
  p.has_r = a.dr != nullptr;
  p.has_y = a.y != nullptr || a.y_saved.codes != nullptr;
  p.dn = p.has_n ? a.dn : a.dx;
  p.dr = p.has_r ? a.dr : a.dx;
  p.r = a.r != nullptr ? a.r : a.r_saved.codes != nullptr ? a.r_saved.codes : a.dx;
  p.y = a.y != nullptr ? a.y : a.y_saved.codes != nullptr ? a.y_saved.codes : a.dx;
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
  f.slices = g.groups < kFinishY ? kFinishY / (int)g.groups : 1;
  const int64_t items = g.groups * shape.chunks;
  const int64_t group_blocks = (g.groups + kGroupWarps - 1) / kGroupWarps * f.channel_blocks;
  if (items > INT32_MAX || group_blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaError_t e = g.bf16 ? launch_type<__nv_bfloat16>(p, (unsigned)items, s) : launch_type<float>(p, (unsigned)items, s);
  if (e != cudaSuccess || p.need == 0) return e;
  if (g.groups <= kFewGroups) return launch_dependent(norm_bwd_finish_kernel, dim3(g.C / kFinishX), dim3(kFinishX, kFinishY), f, s);
  e = launch_dependent(norm_bwd_groups_kernel, dim3((unsigned)group_blocks), dim3(32, kGroupWarps), f, s);
  if (e == cudaSuccess && (a.dweight != nullptr || a.dpost_weight != nullptr))
    e = launch_dependent(norm_bwd_weights_kernel, dim3(f.channel_blocks), dim3(32, 32), f, s);
  return e;
}

}  // namespace ssta
