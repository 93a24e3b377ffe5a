// Attention over the paged 4-bit key/value cache.
//
//   o = U^T sum_t p_t v_t / sum_t p_t,   p_t = exp(scale (T q) . k_t),   k_t, v_t = code * group scale
//
// for every new row of every sequence, T and U the rotations that the cache stores keys and values in.
// Bound by HBM for single tokens (the cache is read once: D + 4 D/G bytes per token and key head) and by
// the tensor pipe and the unpacking for many rows.
//
// A CTA takes 8 NT query rows (row = new token x query head of one key head) and a part of the length.
// Its warps are independent: each takes every W-th tile of 32 tokens through a ring of its own in shared
// memory (one bulk copy per tile), with its own running maximum, and the warps' sums are joined at the
// end. Tokens lie on the m axis of m16n8k16 MMAs, query rows on n, so that a few rows waste no tensor work:
//   S^T = K Q^T    the key codes are the A operand as they are: a nibble u = q + 8 masked in place is the
//                  binary16 subnormal u 2^-24 (bits 0..3) or 16 u 2^-24 (bits 4..7, Q pre-divided by 16),
//                  five logic operations for eight codes and no conversion; -8 sum q enters as the
//                  accumulator's start. One accumulator per group, scaled in fp32.
//   P              fp32 exponentials against a reference that is only raised when a logit passes it by
//                  2^8, binary16 towards the MMA, transposed by movmatrix, times the value scales.
//   O^T = V^T P    value codes of two tokens paired by prmt, again as subnormals; -8 sum P from one MMA
//                  with ones per group.
// Roundings below 32 bits: the rotated query (binary16 after an exact power-of-two scaling per row) and
// P and P * scale (binary16, 2^-11 / 2 each); sums, maxima and logits are fp32. bf16 for P would round at
// 2^-8 / 2, as coarse as the bf16 output itself.
#include <algorithm>

#include "kv4.cuh"

namespace rotb {
namespace {

__device__ int g_kv4_attn_error = 0;

constexpr int W = 4;              // warps of a CTA
constexpr int CTA = 32 * W;
constexpr int P_SHIFT = 7;        // P is held as p 2^7, p <= 2^8 of the reference: below 2^15
constexpr float NINF = -__builtin_huge_valf();

struct Params {
  Kv4View c;
  const void* q;
  int64_t q_token, q_head;
  __nv_bfloat16* out;
  float* part;     // [T * Hq][splits][D]
  float* part_ml;  // [T * Hq][splits][2]
  int Hq, share, causal, window, chunks, splits;
  float scale_log2;  // softmax scale * log2 e
  float norm;        // 1 / sqrt(D)
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, const float (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// offset nibbles u = q + 8 of two packed halves as binary16 subnormals: bits 0..3 and bits 4..7
__device__ __forceinline__ uint32_t lo_nib(uint32_t w) { return (w & 0x000F000Fu) ^ 0x00080008u; }
__device__ __forceinline__ uint32_t hi_nib(uint32_t w) { return (w & 0x00F000F0u) ^ 0x00800080u; }

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t max_half2(uint32_t a, uint32_t b) {  // drops NaN
  const __half2 h = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// n 32-bit words from shared memory with the widest loads
template <int N>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                   : "r"(addr + 4 * i));
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  } else {
    static_assert(N == 1);
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
  }
}

// Waits for a stage's copy, for at most about a second; false where it gave up
__device__ __forceinline__ bool wait_full(uint32_t bar, uint32_t parity) {
  uint32_t done = 0;
  unsigned long long t0 = 0;
  while (true) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tmbarrier.try_wait.parity.shared::cta.b64 q, [%1], %2;\n\tselp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (done) return true;
    unsigned long long t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    if (!t0) t0 = t;
    if (t - t0 > 1000000000ull) return false;
  }
}

// The NG binary16 scales of a token (keys), as fp32; an infinite scale (its codes are 0) becomes NaN
template <int NG>
__device__ __forceinline__ void key_scales(uint32_t addr, float (&s)[NG]) {
  if constexpr (NG == 1) {
    uint16_t h;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(addr));
    s[0] = __half2float(__ushort_as_half(h));
  } else {
    uint32_t w[NG / 2];
    lds<NG / 2>(addr, w);
#pragma unroll
    for (int i = 0; i < NG; ++i) s[i] = __half2float(__ushort_as_half((uint16_t)(w[i / 2] >> (16 * (i & 1)))));
  }
#pragma unroll
  for (int i = 0; i < NG; ++i) s[i] = fmaf(s[i], 0.0f, s[i]);
}

constexpr int stages_of(int D) { return D == 256 ? 2 : D == 128 ? 3 : 4; }

template <int D, int NG, int NT>
struct Lay {
  static constexpr int TILE = kv4_tile_bytes(D, NG);
  static constexpr int ST = stages_of(D);
  static constexpr int ROWS = 8 * NT;
  static constexpr int OUT = ROWS * (D + 4) * 4;               // a warp's O at the end, in place of its ring
  static constexpr int RING = ST * TILE > OUT ? ST * TILE : OUT;
  static constexpr int QF = NT * (D / 32) * 32 * 16;           // B fragments of Q: [nt][j][lane] 16 bytes
  static constexpr int BIAS = ROWS * NG * 4;                   // -8 2^-24 sum q' per row and group
  static constexpr int O_Q = W * RING;
  static constexpr int O_BIAS = O_Q + QF;
  static constexpr int O_FAC = O_BIAS + BIAS;                  // per row: logit factor
  static constexpr int O_ML = O_FAC + ROWS * 4;                // [W][ROWS][2]
  static constexpr int O_BAR = O_ML + W * ROWS * 8;
  static constexpr int SMEM = O_BAR + W * ST * 8;
};

// Final row: joined sums o (lane's D/32 coordinates) over l, back through U^T, to bf16
template <int D>
__device__ __forceinline__ void finish_row(const Params& p, float (&o)[D / 32], float l, int64_t row, int lane) {
  constexpr int V = D / 32;
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;  // nothing seen: zeros (a NaN sum stays)
  float scale = inv;
  if (p.c.v_rot) {
    kv4_fwht<V, 32>(o, lane);
    scale *= p.norm;
    if (p.c.v_sign) {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const uint32_t w = __ldg(p.c.v_sign + (lane * V + i) / 2);
        o[i] = kv4_signed(o[i], w, 0);
        o[i + 1] = kv4_signed(o[i + 1], w, 1);
      }
    }
  }
  uint32_t w[V / 2];
#pragma unroll
  for (int i = 0; i < V; i += 2) w[i / 2] = kv4_pack_bf16(o[i] * scale, o[i + 1] * scale);
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + row * D + lane * V);
  if constexpr (V == 2) dst[0] = w[0];
  else if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D, int NG, int NT, bool QF32>
__global__ void __launch_bounds__(CTA) attention_kernel(const __grid_constant__ Params p) {
  using L = Lay<D, NG, NT>;
  constexpr int J = D / 32, JG = J / NG, V = D / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::O_BAR) + warp * L::ST;
  if (lane == 0) {
    for (int s = 0; s < L::ST; ++s)
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(bars + s)) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // blockIdx.x = ((b * chunks + chunk) * heads + h) * splits + split
  uint32_t id = blockIdx.x;
  const int split = (int)(id % (uint32_t)p.splits);
  id /= (uint32_t)p.splits;
  const int h = (int)(id % (uint32_t)p.c.heads);
  id /= (uint32_t)p.c.heads;
  int chunk = (int)(id % (uint32_t)p.chunks);
  const int b = (int)(id / (uint32_t)p.chunks);

  int64_t first, first_pos;
  const int n_new = kv4_new_rows(p.c, b, &first, &first_pos);
  const int n_rows = n_new * p.share;
  const int len = max(p.c.lens[b], 0);
  const int pos0 = (int)first_pos;  // position of the sequence's first new token
  uint32_t phases = 0;

  const uint32_t ring = smem_u32(smem) + warp * L::RING;
  float* qs_fac = reinterpret_cast<float*>(smem + L::O_FAC);
  float* qs_bias = reinterpret_cast<float*>(smem + L::O_BIAS);
  uint32_t* qs = reinterpret_cast<uint32_t*>(smem + L::O_Q);
  float* ml = reinterpret_cast<float*>(smem + L::O_ML);

  // (chunks beyond the launch's: only where the caller's max_new was too small)
  for (; chunk * L::ROWS < n_rows; chunk += p.chunks) {
    const int row0 = chunk * L::ROWS;
    // ---- the tokens that this CTA's rows see: [low, high)
    const int last = min(row0 + L::ROWS, n_rows) - 1;
    const int pos_a = pos0 + row0 / p.share, pos_z = pos0 + last / p.share;
    int high = len, low = 0;
    if (p.causal) high = min(len, max(pos_z + 1, 0));
    if (p.window) low = max(0, pos_a - p.window + 1);
    const int tile_a = low >> 5, tiles = high > low ? ((high + 31) >> 5) - tile_a : 0;
    const int from = (int)((int64_t)tiles * split / p.splits), to = (int)((int64_t)tiles * (split + 1) / p.splits);
    const int count = to - from > warp ? (to - from - warp + W - 1) / W : 0;  // this warp's tiles
    const int tile0 = tile_a + from + warp;

    int64_t my_at = -1;   // lane's tile address out of the next 32
    uint32_t have = 0;    // stages that hold a tile
    auto issue = [&](int i) {  // tile i of this warp into stage i % ST
      if ((i & 31) == 0) {
        const int mine = i + lane;
        my_at = -1;
        if (mine < count) {
          my_at = kv4_tile_at(p.c, b, tile0 + (int64_t)mine * W, h);
          if (my_at < 0) atomicExch(&g_kv4_attn_error, (int)ROT_EINVAL);
        }
      }
      const int64_t at = __shfl_sync(0xffffffffu, my_at, i & 31);
      const int s = i % L::ST;
      if (at < 0) {
        have &= ~(1u << s);
        return;
      }
      have |= 1u << s;
      if (lane == 0) {
        const uint32_t bar = smem_u32(bars + s);
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(L::TILE) : "memory");
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         ring + s * L::TILE),
                     "l"(p.c.data + at), "r"(L::TILE), "r"(bar)
                     : "memory");
      }
    };
    for (int i = 0; i < L::ST && i < count; ++i) issue(i);

    // ---- the CTA's query rows: rotate, scale to binary16 by a power of two, B fragment order
    for (int rr = warp; rr < L::ROWS; rr += W) {
      const int row = row0 + rr;
      float v[V];
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = 0.0f;
      if (row < n_rows) {
        const int64_t at = (first + row / p.share) * p.q_token + ((int64_t)h * p.share + row % p.share) * p.q_head + lane * V;
        if constexpr (QF32) {
          const float2* src = reinterpret_cast<const float2*>(static_cast<const float*>(p.q) + at);
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            const float2 x = __ldg(src + i);
            v[2 * i] = x.x;
            v[2 * i + 1] = x.y;
          }
        } else {
          const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.q) + at);
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            const uint32_t x = __ldg(src + i);
            v[2 * i] = __uint_as_float(x << 16);
            v[2 * i + 1] = __uint_as_float(x & 0xffff0000u);
          }
        }
      }
      float fac = p.scale_log2;
      if (p.c.k_rot) {
        if (p.c.k_sign) {
#pragma unroll
          for (int i = 0; i < V; i += 2) {
            const uint32_t w = __ldg(p.c.k_sign + (lane * V + i) / 2);
            v[i] = kv4_signed(v[i], w, 0);
            v[i + 1] = kv4_signed(v[i + 1], w, 1);
          }
        }
        kv4_fwht<V, 32>(v, lane);
        fac *= p.norm;
      }
      // largest magnitude to [2^14, 2^15): an exact scaling, so that small queries keep their bits
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
      for (int x = 1; x < 32; x *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
      const int e = m > 0.0f ? min(max(141 - (int)(__float_as_uint(m) >> 23), -100), 100) : 0;
      const float up = __uint_as_float((uint32_t)(127 + e) << 23);
      // 2^24 of the subnormal codes and 2^-e, in two steps that stay in range
      fac = fac * 16777216.0f * __uint_as_float((uint32_t)(127 - e) << 23);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int d = lane * V + i, in = d & 7;  // coordinate 32 j + 8 c + in
        const bool odd = in & 1;
        const __half q16 = __float2half_rn(v[i] * up * (odd ? 0.0625f : 1.0f));
        sum += __half2float(q16) * (odd ? 16.0f : 1.0f);
        // fragment register in / 2 of 0..3 by pairs (0,4) (1,5) (2,6) (3,7); half by in >= 4
        const int at = ((((rr >> 3) * J + (d >> 5)) * 32 + (rr & 7) * 4 + ((d >> 3) & 3)) * 4 + (in & 3)) * 2 + (in >> 2);
        reinterpret_cast<__half*>(qs)[at] = q16;
      }
#pragma unroll
      for (int x = 1; x < 32 / NG; x *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      if (lane % (32 / NG) == 0) qs_bias[rr * NG + lane / (32 / NG)] = sum * (-8.0f / 16777216.0f);
      if (lane == 0) qs_fac[rr] = fac;
    }
    __syncthreads();

    // ---- per thread: columns 2c, 2c + 1 of each n-tile
    float fac[NT][2], ref[NT][2], sum[NT][2];
    int seen_hi[NT][2], seen_lo[NT][2], all_hi = high, all_lo = low;
    float o[NT][2 * J][4], ones[NT][NG][4], bias[NT][NG][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int rr = nt * 8 + 2 * c + k, row = row0 + rr;
        fac[nt][k] = qs_fac[rr];
        ref[nt][k] = NINF;
        sum[nt][k] = 0.0f;
        seen_hi[nt][k] = high;
        seen_lo[nt][k] = 0;
        if (row < n_rows) {
          const int pos = pos0 + row / p.share;
          if (p.causal) seen_hi[nt][k] = min(high, pos + 1);
          if (p.window) seen_lo[nt][k] = max(0, pos - p.window + 1);
          all_hi = min(all_hi, seen_hi[nt][k]);
          all_lo = max(all_lo, seen_lo[nt][k]);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) bias[nt][g][k] = qs_bias[rr * NG + g];
      }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int m = 0; m < 2 * J; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][m][i] = 0.0f;
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) ones[nt][g][i] = 0.0f;
    }
#pragma unroll
    for (int x = 1; x < 4; x *= 2) {
      all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, x));
      all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, x));
    }
    int vexp = -15;  // value scales are at most 2^vexp and enter the MMA as s 2^-vexp

    for (int i = 0; i < count; ++i) {
      const int s = i % L::ST;
      if (!(have >> s & 1)) {  // no such page: nothing of it is seen
        if (i + L::ST < count) issue(i + L::ST);
        continue;
      }
      if (!__all_sync(0xffffffffu, wait_full(smem_u32(bars + s), (phases >> s) & 1))) {
        // the copies behind this one get the same time, then the launch's outputs are given up
        for (int t = 0; t < L::ST; ++t)
          if (have >> t & 1) wait_full(smem_u32(bars + t), (phases >> t) & 1);
        if (lane == 0) atomicExch(&g_kv4_attn_error, (int)ROT_ETIMEOUT);
        break;
      }
      phases ^= 1u << s;
      have &= ~(1u << s);
      const uint32_t tile = ring + s * L::TILE;
      const int tok0 = (tile0 + i * W) * 32;
#pragma unroll 1
      for (int sub = 0; sub < 2; ++sub) {
        const int tk = tok0 + 16 * sub;
        if (tk >= high || tk + 16 <= low) continue;
        const bool edge = tk < all_lo || tk + 16 > all_hi;
        // ---- S^T: tokens r, r + 8 by columns 2c, 2c + 1
        float S[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) S[nt][k] = 0.0f;
        uint32_t k0[J], k1[J];
        lds<J>(tile + (16 * sub + r) * (D / 2) + c * (D / 8), k0);
        lds<J>(tile + (16 * sub + r + 8) * (D / 2) + c * (D / 8), k1);
        float s0[NG], s1[NG];
        key_scales<NG>(tile + 32 * D + (16 * sub + r) * (2 * NG), s0);
        key_scales<NG>(tile + 32 * D + (16 * sub + r + 8) * (2 * NG), s1);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float acc[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            acc[nt][0] = acc[nt][2] = bias[nt][g][0];
            acc[nt][1] = acc[nt][3] = bias[nt][g][1];
          }
#pragma unroll
          for (int jj = 0; jj < JG; ++jj) {
            const int j = g * JG + jj;
            const uint32_t a0[4] = {lo_nib(k0[j]), lo_nib(k1[j]), hi_nib(k0[j]), hi_nib(k1[j])};
            const uint32_t x0 = k0[j] >> 8, x1 = k1[j] >> 8;
            const uint32_t a1[4] = {lo_nib(x0), lo_nib(x1), hi_nib(x0), hi_nib(x1)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint32_t qf[4];
              lds<4>(smem_u32(qs) + ((nt * J + j) * 32 + lane) * 16, qf);
              mma(acc[nt], a0, qf[0], qf[1], acc[nt]);
              mma(acc[nt], a1, qf[2], qf[3], acc[nt]);
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            S[nt][0] = fmaf(s0[g], acc[nt][0], S[nt][0]);
            S[nt][1] = fmaf(s0[g], acc[nt][1], S[nt][1]);
            S[nt][2] = fmaf(s1[g], acc[nt][2], S[nt][2]);
            S[nt][3] = fmaf(s1[g], acc[nt][3], S[nt][3]);
          }
        }
        // ---- value scales of the pairs c, c + 4 of this half tile
        uint32_t vs[2][NG];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          lds<NG>(tile + 32 * D + 64 * NG + (8 * sub + 4 * hh + c) * (4 * NG), vs[hh]);
          if (edge) {  // tokens outside the sequence hold whatever was there
            const int t = tk + 8 * hh + 2 * c;
            const uint32_t keep = (t >= low && t < high ? 0xffffu : 0u) | (t + 1 >= low && t + 1 < high ? 0xffff0000u : 0u);
#pragma unroll
            for (int g = 0; g < NG; ++g) vs[hh][g] &= keep;
          }
        }
        uint32_t big = vs[0][0];
#pragma unroll
        for (int g = 0; g < NG; ++g) big = max_half2(big, max_half2(vs[0][g], vs[1][g]));
        // ---- logits; those outside a row's reach vanish
        float top = NINF;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            S[nt][k] *= fac[nt][k & 1];
            if (edge) {
              const int t = tk + r + 8 * (k >> 1);
              if (t >= seen_hi[nt][k & 1] || t < seen_lo[nt][k & 1]) S[nt][k] = NINF;
            }
            top = fmaxf(top, S[nt][k] - ref[nt][k & 1]);
          }
        const __half2 big2 = *reinterpret_cast<const __half2*>(&big);
        const float bigf = fmaxf(__low2float(big2), __high2float(big2));
        const float vtop = __uint_as_float((uint32_t)(127 + vexp) << 23);
        if (__any_sync(0xffffffffu, top > 8.0f || bigf > vtop)) {
          // raise the references of all rows to their largest logit so far, and the values' exponent
          float bm = bigf;
#pragma unroll
          for (int x = 1; x < 32; x *= 2) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, x));
          const int be = min(max((int)(__float_as_uint(bm) >> 23) - 126, -14), 16);  // bm <= 2^be
          const int nexp = max(vexp, be);
          const float down = __uint_as_float((uint32_t)(127 + vexp - nexp) << 23);
          vexp = nexp;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float m = fmaxf(S[nt][k], S[nt][k + 2]);
#pragma unroll
              for (int x = 4; x < 32; x *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
              m = fmaxf(m, ref[nt][k]);
              const float f = ref[nt][k] == NINF ? 0.0f : ex2(ref[nt][k] - m);
              ref[nt][k] = m;
              sum[nt][k] *= f;
              const float fo = f * down;
#pragma unroll
              for (int t = 0; t < 2 * J; ++t) {
                o[nt][t][k] *= fo;
                o[nt][t][k + 2] *= fo;
              }
#pragma unroll
              for (int g = 0; g < NG; ++g) {
                ones[nt][g][k] *= fo;
                ones[nt][g][k + 2] *= fo;
              }
            }
        }
        // ---- P 2^7 towards the MMA's B operand: [column][token]
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // a row that has seen nothing yet has ref -inf: all its logits here are -inf too
            const float at = fmaxf(ref[nt][k & 1], -3.0e38f);
            e[k] = ex2(S[nt][k] - at + (float)P_SHIFT);
            sum[nt][k & 1] += e[k];
          }
          pb[nt][0] = transpose8(pack_half(e[0], e[1]));
          pb[nt][1] = transpose8(pack_half(e[2], e[3]));
        }
        const __half vdown1 = __float2half_rn(__uint_as_float((uint32_t)(127 - vexp) << 23));
        const uint32_t vdown = (uint32_t)__half_as_ushort(vdown1) * 0x00010001u;
        // ---- O^T
        uint32_t vw[2][J];  // [h]: blocks by token b = 0, then b = 1
        lds<J>(tile + 16 * D + sub * (8 * D) + (r * 4 + c) * (D / 8), vw[0]);
        lds<J>(tile + 16 * D + sub * (8 * D) + 4 * D + (r * 4 + c) * (D / 8), vw[1]);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          uint32_t pv[NT][2];
          const uint32_t sv[2] = {mul_half2(vs[0][g], vdown), mul_half2(vs[1][g], vdown)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              pv[nt][hh] = mul_half2(pb[nt][hh], sv[hh]);
              if (edge) {  // a NaN or infinite scale of a token that this row does not see
                const uint32_t x = pb[nt][hh];
                pv[nt][hh] &= ((x & 0x7fffu) ? 0xffffu : 0u) | ((x & 0x7fff0000u) ? 0xffff0000u : 0u);
              }
            }
          const uint32_t one[4] = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma(ones[nt][g], one, pv[nt][0], pv[nt][1], ones[nt][g]);
#pragma unroll
          for (int jj = 0; jj < JG; ++jj) {
            const int j = g * JG + jj;
            const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
            uint32_t xa = prmt(vw[0][j / 2], vw[0][J / 2 + j / 2], sel);
            uint32_t xb = prmt(vw[1][j / 2], vw[1][J / 2 + j / 2], sel);
            const uint32_t a0[4] = {lo_nib(xa), hi_nib(xa), lo_nib(xb), hi_nib(xb)};
            xa >>= 8;
            xb >>= 8;
            const uint32_t a1[4] = {lo_nib(xa), hi_nib(xa), lo_nib(xb), hi_nib(xb)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma(o[nt][2 * j], a0, pv[nt][0], pv[nt][1], o[nt][2 * j]);
              mma(o[nt][2 * j + 1], a1, pv[nt][0], pv[nt][1], o[nt][2 * j + 1]);
            }
          }
        }
      }
      __syncwarp();
      if (i + L::ST < count) issue(i + L::ST);
    }

    // ---- this warp's sums into shared memory (its ring is drained), then the CTA's join
    float* mine = reinterpret_cast<float*>(smem + warp * L::RING);
    const float back = __uint_as_float((uint32_t)(127 + vexp - P_SHIFT) << 23);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float l = sum[nt][k];
#pragma unroll
        for (int x = 4; x < 32; x *= 2) l += __shfl_xor_sync(0xffffffffu, l, x);
        const int rr = nt * 8 + 2 * c + k;
        if (r == 0) {
          ml[(warp * L::ROWS + rr) * 2] = ref[nt][k];
          ml[(warp * L::ROWS + rr) * 2 + 1] = l * (1.0f / (1 << P_SHIFT));
        }
#pragma unroll
        for (int t = 0; t < 2 * J; ++t) {
          const float off = 8.0f * ones[nt][t / 2 / JG][k];
          const int d = 32 * (t / 2) + 4 * r + 2 * (t & 1);
          mine[rr * (D + 4) + d] = (o[nt][t][k] * 16777216.0f - off) * back;
          mine[rr * (D + 4) + d + 1] = (o[nt][t][k + 2] * 1048576.0f - off) * back;
        }
      }
    __syncthreads();
    for (int rr = warp; rr < L::ROWS; rr += W) {
      const int row = row0 + rr;
      if (row >= n_rows) continue;
      float m = NINF, l = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) m = fmaxf(m, ml[(w * L::ROWS + rr) * 2]);
      float sum_o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) sum_o[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float mw = ml[(w * L::ROWS + rr) * 2];
        const float f = mw == NINF ? 0.0f : ex2(mw - m);
        const float lw = ml[(w * L::ROWS + rr) * 2 + 1];
        if (mw == NINF && lw == 0.0f) continue;
        const float g = mw == NINF ? 1.0f : f;  // only NaN logits so far: keep them
        l += lw * g;
        const float* src = reinterpret_cast<const float*>(smem + w * L::RING) + rr * (D + 4) + lane * V;
#pragma unroll
        for (int i = 0; i < V; ++i) sum_o[i] = fmaf(src[i], g, sum_o[i]);
      }
      const int64_t out_row = (first + row / p.share) * p.Hq + (int64_t)h * p.share + row % p.share;
      if (p.splits == 1) {
        finish_row<D>(p, sum_o, l, out_row, lane);
      } else {
        float* dst = p.part + (out_row * p.splits + split) * D + lane * V;
#pragma unroll
        for (int i = 0; i < V; ++i) dst[i] = sum_o[i];
        if (lane == 0) {
          p.part_ml[(out_row * p.splits + split) * 2] = m;
          p.part_ml[(out_row * p.splits + split) * 2 + 1] = l;
        }
      }
    }
    // the ring held sums: order them before the next chunk's copies into it
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
  }
}

// Joins the parts of a row: one warp per (new token, query head).
template <int D>
__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ Params p) {
  constexpr int V = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= p.c.T * p.Hq) return;
  if (kv4_seq_of(p.c, row / p.Hq) < 0) return;  // behind the last sequence: left as it was
  const float* ml = p.part_ml + row * p.splits * 2;
  float m = NINF;
  for (int s = lane; s < p.splits; s += 32) m = fmaxf(m, ml[2 * s]);
#pragma unroll
  for (int x = 1; x < 32; x *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  float l = 0.0f, o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.0f;
  for (int s = 0; s < p.splits; ++s) {
    const float ms = ml[2 * s], ls = ml[2 * s + 1];
    if (ms == NINF && ls == 0.0f) continue;
    const float f = ms == NINF ? 1.0f : ex2(ms - m);
    l += ls * f;
    const float* src = p.part + (row * p.splits + s) * D + lane * V;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = fmaf(src[i], f, o[i]);
  }
  finish_row<D>(p, o, l, row, lane);
}

template <class K>
rot_status launch(K kernel, int64_t ctas, int threads, int smem, cudaStream_t s, const Params& p) {
  if (ctas > 0x7fffffff) return set_error(ROT_EUNSUPPORTED, "kv4_attention: too many rows for one launch");
  if (smem > 48 * 1024) ROT_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = pdl_default() ? 1 : 0;
  ROT_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, p));
  return ROT_OK;
}

template <int D, int NG, int NT>
rot_status run(const Params& p, bool q_f32, cudaStream_t s) {
  const int64_t ctas = (int64_t)p.c.B * p.chunks * p.c.heads * p.splits;
  constexpr int smem = Lay<D, NG, NT>::SMEM;
  rot_status st = q_f32 ? launch(attention_kernel<D, NG, NT, true>, ctas, CTA, smem, s, p)
                        : launch(attention_kernel<D, NG, NT, false>, ctas, CTA, smem, s, p);
  if (st || p.splits == 1) return st;
  return launch(combine_kernel<D>, (p.c.T * p.Hq + 3) / 4, 128, 0, s, p);
}

template <int D, int NG>
rot_status run_rows(const Params& p, bool q_f32, int rows, cudaStream_t s) {
  if constexpr (D < 256) {
    if (rows > 8) return run<D, NG, 2>(p, q_f32, s);
  }
  return run<D, NG, 1>(p, q_f32, s);
}

}  // namespace

Kv4Split kv4_split(int D, int B, int heads, int share, int window, int64_t max_new, int64_t max_len, int sms) {
  Kv4Split sp{};
  if (window > 0) max_len = std::min(max_len, max_new + window);
  const int64_t rows = max_new * share;
  sp.rows = rows > 8 && D < 256 ? 16 : 8;
  sp.chunks = (int)std::min<int64_t>(std::max<int64_t>((rows + sp.rows - 1) / sp.rows, 1), 1 << 20);
  const int64_t units = std::max<int64_t>((int64_t)B * heads * sp.chunks, 1);
  const int64_t tiles = (max_len + KV4_TILE - 1) / KV4_TILE;
  const int64_t want = (8 * (int64_t)sms + units - 1) / units;   // CTAs that fill the GPU a few times over
  const int64_t most = (tiles + 4 * W - 1) / (4 * W);            // at least four tiles to a warp
  sp.splits = (int)std::min<int64_t>(std::max<int64_t>(std::min(want, most), 1), 256);
  return sp;
}

rot_status kv4_attention_launch(const Kv4View& c, int D, int NG, const Kv4Query& q, const Kv4Split& sp, cudaStream_t s) {
  Params p{};
  p.c = c;
  p.q = q.q;
  p.q_token = q.q_token;
  p.q_head = q.q_head;
  p.out = static_cast<__nv_bfloat16*>(q.out);
  p.part = q.partial;
  p.part_ml = q.partial ? q.partial + c.T * q.Hq * sp.splits * D : nullptr;
  p.Hq = q.Hq;
  p.share = q.Hq / c.heads;
  p.causal = q.causal;
  p.window = q.window;
  p.chunks = sp.chunks;
  p.splits = sp.splits;
  p.scale_log2 = q.scale * 1.4426950408889634f;
  p.norm = (float)(1.0 / sqrt((double)D));
  const bool f32 = q.q_dtype == ROT_F32;
  switch (D * 16 + NG) {
    case 64 * 16 + 2: return run_rows<64, 2>(p, f32, sp.rows, s);
    case 64 * 16 + 1: return run_rows<64, 1>(p, f32, sp.rows, s);
    case 128 * 16 + 4: return run_rows<128, 4>(p, f32, sp.rows, s);
    case 128 * 16 + 2: return run_rows<128, 2>(p, f32, sp.rows, s);
    case 128 * 16 + 1: return run_rows<128, 1>(p, f32, sp.rows, s);
    case 256 * 16 + 8: return run_rows<256, 8>(p, f32, sp.rows, s);
    case 256 * 16 + 4: return run_rows<256, 4>(p, f32, sp.rows, s);
    case 256 * 16 + 2: return run_rows<256, 2>(p, f32, sp.rows, s);
    case 256 * 16 + 1: return run_rows<256, 1>(p, f32, sp.rows, s);
    default: return set_error(ROT_EUNSUPPORTED, "kv4_attention: no kernel for this D and G");
  }
}

rot_status kv4_attention_fetch_device_error() {
  int v = 0;
  ROT_CUDA_TRY(cudaMemcpyFromSymbol(&v, g_kv4_attn_error, sizeof(int)));
  if (v) {
    int z = 0;
    ROT_CUDA_TRY(cudaMemcpyToSymbol(g_kv4_attn_error, &z, sizeof(int)));
    return set_error((rot_status)v, v == ROT_ETIMEOUT ? "a bounded wait in kv4_attention gave up"
                                                      : "kv4_attention: a page table named no page of the cache for a token");
  }
  return ROT_OK;
}

}  // namespace rotb
