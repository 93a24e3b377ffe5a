// Writing the paged 4-bit key/value cache (rotate, quantise, pack, place) and reading it back.
//
// One row (a token's key or value of one head) is D/32 lanes of 32 coordinates: a lane holds block j of
// the tile layout (kv4.cuh), so a quantisation group of 32 needs no shuffle, the lowest five stages of
// the Walsh-Hadamard transform run in registers, and the rest are one shuffle per value and stage.
// A warp takes 1024/D consecutive tokens of one head, so that the pieces of eight neighbouring tokens
// which the value layout interleaves leave in one store instruction.
// Both kernels are bound by HBM traffic (rows in or out at full width, codes at 4 bits).
#include "kv4.cuh"

namespace rotb {
namespace {

__device__ int g_kv4_cache_error = 0;

constexpr int CTA = 128;

// 32 coordinates from global memory as fp32
template <bool F32>
__device__ __forceinline__ void load32(const void* base, int64_t at, float (&v)[32]) {
  if constexpr (F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 x = __ldg(p + i);
      v[4 * i] = x.x;
      v[4 * i + 1] = x.y;
      v[4 * i + 2] = x.z;
      v[4 * i + 3] = x.w;
    }
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 x = __ldg(p + i);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
        v[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    }
  }
}

template <bool F32>
__device__ __forceinline__ void store32(void* base, int64_t at, const float (&v)[32]) {
  if constexpr (F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
    uint4* p = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = make_uint4(kv4_pack_bf16(v[8 * i], v[8 * i + 1]), kv4_pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                        kv4_pack_bf16(v[8 * i + 4], v[8 * i + 5]), kv4_pack_bf16(v[8 * i + 6], v[8 * i + 7]));
  }
}

__device__ __forceinline__ void apply_signs(float (&v)[32], const uint32_t* sign, int j) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t w = __ldg(sign + 16 * j + i);
    v[2 * i] = kv4_signed(v[2 * i], w, 0);
    v[2 * i + 1] = kv4_signed(v[2 * i + 1], w, 1);
  }
}

// A row's place; a page outside the cache is an error of the call's data.
__device__ __forceinline__ Kv4Slot find(const Kv4View& c, int64_t row, int h) {
  const Kv4Slot p = kv4_slot_of(c, row, h);
  if (p.pos >= 0 && p.at < 0) atomicExch(&g_kv4_cache_error, (int)ROT_EINVAL);
  return p;
}

// Coordinate d of T x for the row at `base`, in 64 bits, by the whole warp.
template <int D, bool F32>
__device__ __noinline__ double exact_coordinate(const void* base, int64_t at, const uint32_t* sign, int d, int lane) {
  constexpr int V = D / 32;
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int k = lane * V + i;
    float x;
    if constexpr (F32) x = __ldg(static_cast<const float*>(base) + at + k);
    else x = __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(base) + at + k));
    if (sign) x = kv4_signed(x, __ldg(sign + k / 2), k & 1);
    sum += (__popc(k & d) & 1) ? -(double)x : (double)x;
  }
#pragma unroll
  for (int m = 1; m < 32; m *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  return sum * (D == 64 ? 0.125 : D == 128 ? 0.08838834764831845 : 0.0625);  // 1 / sqrt(D)
}

// The decision itself, on the rotated value rounded once to fp32: clamp(round_half_away(y / s)) + 8, halves
// away from zero by the floor of fp32(|y / s| + 1/2)
__device__ __forceinline__ uint32_t decide(float y, float s) {
  const float v = __fdiv_rn(y, s);
  const float q = fminf(floorf(__fadd_rn(fabsf(v), 0.5f)), 7.0f);
  return (uint32_t)(8 + (int)copysignf(q, v));
}

// Symmetric absmax int4 codes of the lane's 32 coordinates z (unnormalised where rotated, y = z norm):
// s = binary16(fp32(max|y| / 7)), q = clamp(round_half_away(fp32(y / s))), decided as if the rotation had
// been done in 64 bits and rounded once to fp32. The fp32 butterfly is off by some 3e-7 of the row's
// largest value, so a decision that stands further than that from its border is taken as it is; the few
// others (codes within 4e-6 of a half, about 8e-6 of them, and scales within 4e-7 of a binary16 midpoint,
// about 1e-3; more where the row's largest value is far above the group's) are taken again from a 64-bit
// sum of their own, by the whole warp. A code that flips moves its value by a whole step, which no
// tolerance on the value can tell from a mistake. A group that holds a NaN, or whose scale overflows,
// keeps that scale and codes of 0. All lanes of the warp enter.
template <int D, int NG, bool F32>
__device__ __forceinline__ void quantise(const float (&z)[32], bool rot, float norm, const void* base, int64_t at,
                                         const uint32_t* sign, int lane, uint32_t (&w)[4], uint16_t* scale) {
  constexpr int J = D / 32, L = J / NG;  // lanes of a row, of a group
  const int j = lane % J;
  float m = fabsf(z[0]);
#pragma unroll
  for (int i = 1; i < 32; ++i) m = kv4_max_nan(m, fabsf(z[i]));
#pragma unroll
  for (int x = 1; x < L; x *= 2) m = kv4_max_nan(m, __shfl_xor_sync(0xffffffffu, m, x));
  float row = m;
#pragma unroll
  for (int x = L; x < J; x *= 2) row = fmaxf(row, __shfl_xor_sync(0xffffffffu, row, x));
  const float n1 = rot ? norm : 1.0f;
  float q7 = __fdiv_rn(m * n1, 7.0f);
  // the row's largest value over the group's; without a rotation z is exact, only the quotient is not
  const float far = m > 0.0f ? (rot ? fminf(row / m, 1e6f) : 1.0f) : 0.0f;
  auto candidates = [&](uint32_t mask, auto&& take) {  // exact values of the marked coordinates of every lane
    uint32_t left;
    while ((left = __ballot_sync(0xffffffffu, mask != 0))) {
      const int src = __ffs(left) - 1;
      const int i = __shfl_sync(0xffffffffu, __ffs(mask) - 1, src);
      const double y = exact_coordinate<D, F32>(base, __shfl_sync(0xffffffffu, at, src), sign, 32 * (src % J) + i, lane);
      if (lane == src) {
        mask &= mask - 1;
        take(i, y);
      }
    }
  };
  if (rot) {
    const float eps = 4e-7f * far;
    const bool near = __half_as_ushort(__float2half_rn(q7 * (1.0f - eps))) != __half_as_ushort(__float2half_rn(q7 * (1.0f + eps)));
    if (__any_sync(0xffffffffu, near)) {
      uint32_t mask = 0;
      if (near)
#pragma unroll
        for (int i = 0; i < 32; ++i) mask |= (fabsf(z[i]) >= m * (1.0f - 2.0f * eps) ? 1u : 0u) << i;
      double big = 0.0;
      candidates(mask, [&](int, double y) { big = fmax(big, fabs(y)); });
#pragma unroll
      for (int x = 1; x < L; x *= 2) big = fmax(big, __shfl_xor_sync(0xffffffffu, big, x));
      if (near) q7 = __fdiv_rn((float)big, 7.0f);
    }
  }
  const __half s16 = __float2half_rn(q7);
  const uint32_t hb = __half_as_ushort(s16);
  const float s = __half2float(s16);
  *scale = (uint16_t)hb;
  const bool ok = s > 0.0f && s <= 65504.0f;
  const float f = ok ? __fdiv_rn(n1, s) : 0.0f;
  constexpr float magic = magic_of_bits(4);
  uint32_t u[32];
  float worst = 0.0f;  // distance from the rounded code: a half is the border
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    float t = __fmaf_rn(z[i], f, magic);
    worst = fmaxf(worst, fabsf(__fmaf_rn(z[i], f, magic - t)));
    u[i] = __float_as_uint(t);
  }
  if (((hb & 0x7fffu) - 0x0400u) >= 0x7800u) {  // zero, subnormal (|y / s| may pass 7.5), infinite or NaN scale
#pragma unroll
    for (int i = 0; i < 32; ++i) u[i] = ok ? code_magic_clamped(z[i], f, 7.0f, magic) : 8u;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    w[k] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[k] |= (u[8 * k + i] & 15u) << (4 * i);
  }
  const float border = 0.5f - 4e-6f * far;
  const bool near = ok && worst >= border;
  if (__any_sync(0xffffffffu, near)) {
    uint32_t mask = 0;
    if (near)
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float t = __fmaf_rn(z[i], f, magic);
        mask |= (fabsf(__fmaf_rn(z[i], f, magic - t)) >= border ? 1u : 0u) << i;
      }
    auto patch = [&](int i, uint32_t code) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i / 8 == k) w[k] = (w[k] & ~(15u << (4 * (i & 7)))) | (code << (4 * (i & 7)));
    };
    if (rot) {
      candidates(mask, [&](int i, double y) { patch(i, decide((float)y, s)); });
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (mask >> i & 1) patch(i, decide(z[i], s));
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] ^= offset_xor_of_bits(4);
}

template <int D, int NG, bool F32>
__global__ void __launch_bounds__(CTA) append_kernel(const Kv4View c, const Kv4Rows in, float norm, int64_t warps) {
  constexpr int J = D / 32, TPW = 32 / J;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, j = lane % J;
  const int64_t wid = (int64_t)blockIdx.x * (CTA / 32) + (threadIdx.x >> 5);
  if (wid >= warps) return;
  // warps: heads fastest, then keys / values, then token groups
  const int h = (int)(wid % c.heads);
  const int64_t rest = wid / c.heads;
  const bool val = rest & 1;
  const int64_t row = (rest >> 1) * TPW + lane / J;
  const void* base = val ? in.v : in.k;
  // (lanes behind the last row take row 0's inputs, and store nothing)
  const int64_t at = (row < c.T ? row : 0) * (val ? in.v_token : in.k_token) + h * (val ? in.v_head : in.k_head);
  float z[32];
  load32<F32>(base, at + 32 * j, z);
  const Kv4Slot p = find(c, row, h);
  const int t = (int)(p.pos & 31);
  const bool rot = val ? c.v_rot : c.k_rot;
  const uint32_t* sign = val ? c.v_sign : c.k_sign;
  if (rot) {
    if (sign) apply_signs(z, sign, j);
    kv4_fwht<32, J>(z, lane);
  }
  uint32_t w[4];
  uint16_t sc;
  quantise<D, NG, F32>(z, rot, norm, base, at, sign, lane, w, &sc);
  // values: lanes j and j ^ 1 swap halves of their words, so that each holds four words of two blocks
  uint32_t o[4];
  if (val) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // word k: pieces r = 2k (low half) and 2k + 1 (high half); the even lane collects r = 2k
      const uint32_t other = __shfl_xor_sync(0xffffffffu, w[k], 1);
      o[k] = (j & 1) ? prmt(other, w[k], 0x7632) : prmt(w[k], other, 0x5410);
    }
  }
  if (p.at < 0) return;
  uint8_t* tile = c.data + p.at;
  if (!val) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<uint32_t*>(tile + t * (D / 2) + k * (D / 8) + j * 4) = w[k];
    if (j % (J / NG) == 0)
      *reinterpret_cast<uint16_t*>(tile + 32 * D + (t * NG + j / (J / NG)) * 2) = sc;
  } else {
    uint8_t* v = tile + 16 * D + (t >> 3) * (4 * D) + ((t & 7) >> 1) * (D / 8) + (t & 1) * (D / 16) + (j >> 1) * 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) *reinterpret_cast<uint32_t*>(v + (2 * k + (j & 1)) * (D / 2)) = o[k];
    if (j % (J / NG) == 0)
      *reinterpret_cast<uint16_t*>(tile + 32 * D + 64 * NG + ((t >> 1) * NG + j / (J / NG)) * 4 + (t & 1) * 2) = sc;
  }
}

template <int D, int NG, bool F32>
__global__ void __launch_bounds__(CTA) read_kernel(const Kv4View c, const Kv4Rows out, float norm, int inverse,
                                                   int64_t warps) {
  constexpr int J = D / 32, TPW = 32 / J;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, j = lane % J;
  const int64_t wid = (int64_t)blockIdx.x * (CTA / 32) + (threadIdx.x >> 5);
  if (wid >= warps) return;
  const int h = (int)(wid % c.heads);
  const int64_t rest = wid / c.heads;
  const bool val = rest & 1;
  const int64_t row = (rest >> 1) * TPW + lane / J;
  const Kv4Slot p = find(c, row, h);
  const int t = (int)(p.pos & 31);
  uint32_t w[4] = {0, 0, 0, 0};
  float s = 0.0f;
  if (p.at >= 0) {
    const uint8_t* tile = c.data + p.at;
    uint16_t hb;
    if (!val) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = *reinterpret_cast<const uint32_t*>(tile + t * (D / 2) + k * (D / 8) + j * 4);
      hb = *reinterpret_cast<const uint16_t*>(tile + 32 * D + (t * NG + j / (J / NG)) * 2);
    } else {
      const uint8_t* v = tile + 16 * D + (t >> 3) * (4 * D) + ((t & 7) >> 1) * (D / 8) + (t & 1) * (D / 16) + j * 2;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = *reinterpret_cast<const uint16_t*>(v + 2 * k * (D / 2)) |
               (uint32_t)*reinterpret_cast<const uint16_t*>(v + (2 * k + 1) * (D / 2)) << 16;
      hb = *reinterpret_cast<const uint16_t*>(tile + 32 * D + 64 * NG + ((t >> 1) * NG + j / (J / NG)) * 4 +
                                              (t & 1) * 2);
    }
    s = __half2float(__ushort_as_half(hb));
  }
  float z[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) z[i] = (float)((int)(w[i / 8] << (28 - 4 * (i % 8))) >> 28) * s;
  if (inverse && (val ? c.v_rot : c.k_rot)) {
    // T^T = D H / sqrt(D)
    kv4_fwht<32, J>(z, lane);
    const uint32_t* sign = val ? c.v_sign : c.k_sign;
    if (sign) apply_signs(z, sign, j);
#pragma unroll
    for (int i = 0; i < 32; ++i) z[i] *= norm;
  }
  if (p.seq >= 0)
    store32<F32>(const_cast<void*>(val ? out.v : out.k),
                 row * (val ? out.v_token : out.k_token) + h * (val ? out.v_head : out.k_head) + 32 * j, z);
}

template <class K, class... A>
rot_status launch(K kernel, int64_t warps, cudaStream_t s, const A&... args) {
  const int64_t ctas = (warps + CTA / 32 - 1) / (CTA / 32);
  if (ctas > 0x7fffffff) return set_error(ROT_EUNSUPPORTED, "kv4: too many rows for one launch");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(CTA);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = pdl_default() ? 1 : 0;
  ROT_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, args...));
  return ROT_OK;
}

template <int D, int NG>
rot_status run_append(const Kv4View& c, const Kv4Rows& in, cudaStream_t s) {
  constexpr int TPW = 1024 / D;
  const int64_t warps = (c.T + TPW - 1) / TPW * 2 * c.heads;
  const float norm = (float)(1.0 / sqrt((double)D));
  return in.dtype == ROT_F32 ? launch(append_kernel<D, NG, true>, warps, s, c, in, norm, warps)
                             : launch(append_kernel<D, NG, false>, warps, s, c, in, norm, warps);
}

template <int D, int NG>
rot_status run_read(const Kv4View& c, const Kv4Rows& out, int inverse, cudaStream_t s) {
  constexpr int TPW = 1024 / D;
  const int64_t warps = (c.T + TPW - 1) / TPW * 2 * c.heads;
  const float norm = (float)(1.0 / sqrt((double)D));
  return out.dtype == ROT_F32 ? launch(read_kernel<D, NG, true>, warps, s, c, out, norm, inverse, warps)
                              : launch(read_kernel<D, NG, false>, warps, s, c, out, norm, inverse, warps);
}

}  // namespace

#define KV4_DISPATCH(D, NG, CALL)                                             \
  switch ((D)*16 + (NG)) {                                                    \
    case 64 * 16 + 2: return CALL(64, 2);                                     \
    case 64 * 16 + 1: return CALL(64, 1);                                     \
    case 128 * 16 + 4: return CALL(128, 4);                                   \
    case 128 * 16 + 2: return CALL(128, 2);                                   \
    case 128 * 16 + 1: return CALL(128, 1);                                   \
    case 256 * 16 + 8: return CALL(256, 8);                                   \
    case 256 * 16 + 4: return CALL(256, 4);                                   \
    case 256 * 16 + 2: return CALL(256, 2);                                   \
    case 256 * 16 + 1: return CALL(256, 1);                                   \
    default: return set_error(ROT_EUNSUPPORTED, "kv4: no kernel for this D and G"); \
  }

rot_status kv4_append_launch(const Kv4View& c, int D, int NG, const Kv4Rows& in, cudaStream_t s) {
#define KV4_CALL(d, n) run_append<d, n>(c, in, s)
  KV4_DISPATCH(D, NG, KV4_CALL)
#undef KV4_CALL
}

rot_status kv4_read_launch(const Kv4View& c, int D, int NG, const Kv4Rows& out, bool inverse, cudaStream_t s) {
#define KV4_CALL(d, n) run_read<d, n>(c, out, inverse ? 1 : 0, s)
  KV4_DISPATCH(D, NG, KV4_CALL)
#undef KV4_CALL
}

rot_status kv4_cache_fetch_device_error() {
  int v = 0;
  ROT_CUDA_TRY(cudaMemcpyFromSymbol(&v, g_kv4_cache_error, sizeof(int)));
  if (v) {
    int z = 0;
    ROT_CUDA_TRY(cudaMemcpyToSymbol(g_kv4_cache_error, &z, sizeof(int)));
    return set_error((rot_status)v, "kv4: a page table named no page of the cache for a token (kv4_append / kv4_read)");
  }
  return ROT_OK;
}

}  // namespace rotb
