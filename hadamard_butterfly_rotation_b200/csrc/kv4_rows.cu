// Attention over the 4-bit cache for many query rows of a key head (chunks of prompts, long drafts): the
// same mathematics as kv4_attention.cu with the products on tcgen05.
//
// A CTA (one per SM) takes 256 query rows of one key head as two tiles of 128 and walks 128 tokens (four cache
// tiles) at a time:
//   S = Q K^T    M = 128 rows, N = 128 tokens, both operands in shared memory (K-major, 128-byte swizzle),
//                S in TMEM; one column block for each row tile
//   P            a softmax warp reads its 32 rows of S from TMEM, one row to a thread, and writes P as binary16
//                over the first half of its columns
//   O += P V     A is P in TMEM, B is V in shared memory as it lies in the cache, tokens by rows of
//                coordinates (N-major); O stays in TMEM and is rescaled only when a row's reference rises by
//                more than 2^8
// Warps 0..7 are the softmax of the two row tiles, 8..11 fetch and unpack (each one cache tile of 32 tokens per
// step, with a bulk copy of its own in flight), warp 12 issues the MMAs. While one row tile is in its softmax, the
// tensor pipe works on the other. The unpacking is paid once for 256 rows.
// Codes become binary16 values code * scale 2^-e, e the exponent of the largest scale of the 32 tokens, so that
// any binary16 scale stays in range: key exponents multiply the logits, value exponents the probabilities.
// Roundings below 32 bits: query, key and value operands and P, 2^-11 / 2 relative each. The order of coordinates
// in a row of Q and K, and of V's columns, is the one in which the unpacked words come; Q is written, and O read,
// in the same order.
#include <algorithm>

#include "kv4_attention.cuh"

namespace rotb {
namespace {

using namespace kv4;

__device__ int g_kv4_rows_error = 0;

constexpr int ROWS = KV4_ROWS, TOK = 128;
constexpr int SOFT = 8, UNP = 4, WARPS = SOFT + UNP + 1, CTA = 32 * WARPS;
constexpr unsigned long long WAIT_NS = 1000000000ull;

template <int D, int NG>
struct Lay {
  static constexpr int KV = TOK * D * 2;               // one stage of K or V
  static constexpr int O_Q = 0;                        // [2 row tiles][D / 64 atoms][128 rows][128 bytes]
  static constexpr int O_K = O_Q + ROWS * D * 2;       // [2 stages][D / 64][128 tokens][128 bytes]
  static constexpr int O_V = O_K + 2 * KV;             // the same; both hold O at the end, fp32 [256][D]
  static constexpr int CODES = 16 * D;                 // packed keys, or values, of a cache tile
  static constexpr int SCALES = 128 * NG;              // its scales
  static constexpr int RAW = 2 * CODES + 2 * SCALES;   // keys, values, two sets of scales
  static constexpr int O_RAW = O_V + 2 * KV;           // [UNP]
  static constexpr int O_FAC = O_RAW + UNP * RAW;      // per row: logit factor
  static constexpr int O_SEEN = O_FAC + ROWS * 4;      // per row: the tokens that it sees
  static constexpr int O_ML = O_SEEN + ROWS * 8;       // per row: reference and sum at the end
  static constexpr int O_EXP = O_ML + ROWS * 8;        // [4 steps][UNP]: 2^key exponent, value exponent
  static constexpr int O_ODD = O_EXP + 4 * UNP * 8;    // [4 steps][UNP][NG]: tokens with NaN or infinite value scales
  static constexpr int O_BAR = O_ODD + 4 * UNP * NG * 4;
  static constexpr int BARS = 2 + 2 + 2 + 2 + 4 + 2 + 2 + 2 + 2 * UNP;
  static constexpr int O_TMEM = O_BAR + BARS * 8;
  static constexpr int SMEM = O_TMEM + 16 + 1024;      // (the base is rounded up to 1024)
  static_assert(O_ODD % 8 == 0 && O_BAR % 8 == 0 && SMEM <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t to, const void* from, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "l"(from),
               "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Bounded wait of a converged warp for the phase of that parity; false (recorded, and told to the CTA's other
// warps) where it gave up.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  const uint32_t addr = smem_u32(bar);
  bool ok = true;
  unsigned long long t0 = 0;
  for (uint32_t it = 0;; ++it) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(addr), "r"(parity)
        : "memory");
    if (done) break;
    __nanosleep(20);
    if ((it & 63) == 63) {
      if (*abort_flag) {
        ok = false;
        break;
      }
      unsigned long long now;
      asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
      if (t0 == 0) t0 = now;
      else if (now - t0 > WAIT_NS) {
        *abort_flag = 1;
        atomicExch(&g_kv4_rows_error, (int)ROT_ETIMEOUT);
        ok = false;
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Shared-memory operand descriptors, 128-byte swizzle. K-major: rows of 64 k, eight of them to an atom of 1024
// bytes (the stride). N-major: rows (one for each k) of 64 n; atoms of eight rows follow at the stride along k, the
// next 64 n at the leading offset.
__device__ __forceinline__ uint64_t desc(uint32_t saddr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(stride >> 4) << 32 | (uint64_t)1u << 46 |
         (uint64_t)2u << 61;
}
// binary16 x binary16 -> fp32, M = 128
constexpr uint32_t idesc(int n, bool b_n_major) {
  return (1u << 4) | (b_n_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(e));
  return e != 0;
}
// (by one thread)
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t (&w)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}

// The eight codes of a word as binary16 code * scale, pairs (0, 4) (1, 5) (2, 6) (3, 7): exact integers out of the
// mantissa of 1024 + u and 1024 + 16 u, then one rounding in the product
__device__ __forceinline__ void unpack(uint32_t w, uint32_t scale2, uint32_t (&v)[4]) {
  const uint32_t x = w >> 8;
  uint32_t t[4];
  t[0] = (w & 0x000F000Fu) ^ 0x64086408u;
  t[1] = (w & 0x00F000F0u) ^ 0x64806480u;
  t[2] = (x & 0x000F000Fu) ^ 0x64086408u;
  t[3] = (x & 0x00F000F0u) ^ 0x64806480u;
  const __half2 off = __half2half2(__ushort_as_half(0xE408)), off16 = __half2half2(__ushort_as_half(0xD480));  // -1032, -72
  const __half2 by16 = __half2half2(__ushort_as_half(0x2C00)), s = *reinterpret_cast<const __half2*>(&scale2);  // 1 / 16
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 u = *reinterpret_cast<const __half2*>(&t[i]);
    const __half2 c = __hmul2(i & 1 ? __hfma2(u, by16, off16) : __hadd2(u, off), s);
    v[i] = *reinterpret_cast<const uint32_t*>(&c);
  }
}

template <int D, int NG, bool QF32>
__global__ void __launch_bounds__(CTA, 1) rows_kernel(const __grid_constant__ Params p) {
  using L = Lay<D, NG>;
  constexpr int J = D / 32, JG = J / NG, V = D / 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + L::O_BAR);  // [2] unpacked keys -> MMA
  uint64_t* kempty = kfull + 2;                                    // [2] S of both row tiles done -> unpackers
  uint64_t* vfull = kempty + 2;                                    // [2]
  uint64_t* vempty = vfull + 2;                                    // [2]
  uint64_t* xfull = vempty + 2;                                    // [4] exponents -> softmax
  uint64_t* sfull = xfull + 4;                                     // [2] S of a row tile -> softmax
  uint64_t* pfull = sfull + 2;                                     // [2] P of a row tile -> MMA
  uint64_t* odone = pfull + 2;                                     // [2] P V of a row tile done -> softmax
  uint64_t* rawk = odone + 2;                                      // [UNP] packed keys and scales
  uint64_t* rawv = rawk + UNP;                                     // [UNP] packed values
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::O_TMEM);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::O_TMEM + 8);
  float* r_fac = reinterpret_cast<float*>(smem + L::O_FAC);
  int2* r_seen = reinterpret_cast<int2*>(smem + L::O_SEEN);
  float2* r_ml = reinterpret_cast<float2*>(smem + L::O_ML);
  float2* exps = reinterpret_cast<float2*>(smem + L::O_EXP);
  uint32_t* odds = reinterpret_cast<uint32_t*>(smem + L::O_ODD);

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&kfull[s], UNP);
      mbar_init(&kempty[s], 1);
      mbar_init(&vfull[s], UNP);
      mbar_init(&vempty[s], 1);
      mbar_init(&sfull[s], 1);
      mbar_init(&pfull[s], 4);
      mbar_init(&odone[s], 1);
    }
    for (int s = 0; s < 4; ++s) mbar_init(&xfull[s], UNP);
    for (int s = 0; s < UNP; ++s) {
      mbar_init(&rawk[s], 1);
      mbar_init(&rawv[s], 1);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == WARPS - 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *tmem_slot;  // columns: S or P of row tile 0, 1 (128 each), O of 0, 1
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
  const int n_rows = n_new * p.share, len = max(p.c.lens[b], 0), pos0 = (int)first_pos;
  uint32_t got = 0;   // tiles that an unpacking warp has fetched: the phase of rawk and rawv
  uint32_t step = 0;  // steps of 128 tokens since the start: what the barriers' phases go by
  bool ok = true;

  // (chunks beyond the launch's: only where the caller's max_new was too small)
  for (; chunk * ROWS < n_rows; chunk += p.chunks) {
    const int row0 = chunk * ROWS, last = min(row0 + ROWS, n_rows) - 1, tiles_q = n_rows - row0 > 128 ? 2 : 1;
    // ---- the tokens that this CTA's rows see: [low, high)
    const int pos_a = pos0 + row0 / p.share, pos_z = pos0 + last / p.share;
    int high = len, low = 0;
    if (p.causal) high = min(len, max(pos_z + 1, 0));
    if (p.window) low = max(0, pos_a - p.window + 1);
    const int step_a = low / TOK, steps = high > low ? (high + TOK - 1) / TOK - step_a : 0;
    const int from = (int)((int64_t)steps * split / p.splits), to = (int)((int64_t)steps * (split + 1) / p.splits);
    const int n = to - from, tok_a = (step_a + from) * TOK;

    // ---- query rows: rotate, scale to binary16 by a power of two, K-major
    for (int rr = warp; rr < tiles_q * 128; rr += WARPS) {
      const int row = row0 + rr;
      float v[V];
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = 0.0f;
      if (row < n_rows) {
        const int64_t at = (first + row / p.share) * p.q_token + ((int64_t)h * p.share + row % p.share) * p.q_head + lane * V;
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          if constexpr (QF32) {
            const float2 x = __ldg(reinterpret_cast<const float2*>(static_cast<const float*>(p.q) + at + i));
            v[i] = x.x;
            v[i + 1] = x.y;
          } else {
            const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.q) + at + i));
            v[i] = __uint_as_float(x << 16);
            v[i + 1] = __uint_as_float(x & 0xffff0000u);
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
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
      for (int x = 1; x < 32; x *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
      const int e = m > 0.0f ? min(max(141 - (int)(__float_as_uint(m) >> 23), -100), 100) : 0;
      const float up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int d = lane * V + i, q8 = d >> 3, place = 2 * (d & 3) + ((d >> 2) & 1);
        uint8_t* at = smem + L::O_Q + (rr >> 7) * (128 * D * 2) + (q8 >> 3) * (128 * 128) + (rr & 127) * 128 +
                      (((q8 & 7) ^ (rr & 7)) << 4) + place * 2;
        *reinterpret_cast<__half*>(at) = __float2half_rn(v[i] * up);
      }
      if (lane == 0) {
        r_fac[rr] = fac * __uint_as_float((uint32_t)(127 - e) << 23);
        int2 seen = make_int2(0, high);  // the tokens that the row sees: [x, y)
        if (row < n_rows) {
          const int pos = pos0 + row / p.share;
          if (p.causal) seen.y = min(high, pos + 1);
          if (p.window) seen.x = max(0, pos - p.window + 1);
        }
        r_seen[rr] = seen;
      }
    }
    fence_async();
    __syncthreads();

    if (warp < SOFT) {
      // ======================= softmax: thread = row
      const int q = warp >> 2, rr = q * 128 + (warp & 3) * 32 + lane;
      const uint32_t lane_at = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t s_at = lane_at + q * 128, o_at = lane_at + 256 + q * D;
      if (q < tiles_q) {
        const float fac = r_fac[rr];
        const int2 seen = r_seen[rr];
        float ref = NINF, sum = 0.0f, vref = -15.0f;
        uint32_t poison = 0;  // groups whose value is NaN
        for (int i = 0; i < n && ok; ++i) {
          const uint32_t g = step + i;
          const int tok = tok_a + i * TOK;
          ok = wait(&xfull[g & 3], (g >> 2) & 1, abort_flag) && wait(&sfull[q], g & 1, abort_flag);
          if (!ok) break;
          tc_after();
          const bool edge = __any_sync(0xffffffffu, tok < seen.x || tok + TOK > seen.y);
          const float2* ex = exps + (g & 3) * UNP;
          float top = NINF, vtop = vref;
          uint32_t s[32];
          auto masked = [&](int c) {
            if (edge) {
              const int lo = seen.x - tok - 32 * c, hi = seen.y - tok - 32 * c;
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (k < lo || k >= hi) s[k] = __float_as_uint(NINF);
            }
          };
          // a row's largest logit (fac < 0 turns a masked one around: masked after the product)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_ld32(s_at + 32 * c, s);
            wait_ld();
            const float f = fac * ex[c].x;
            vtop = fmaxf(vtop, ex[c].y);
#pragma unroll
            for (int k = 0; k < 32; ++k) s[k] = __float_as_uint(__uint_as_float(s[k]) * f);
            masked(c);
#pragma unroll
            for (int k = 0; k < 32; k += 2) top = fmaxf(top, fmaxf(__uint_as_float(s[k]), __uint_as_float(s[k + 1])));
          }
          if (__any_sync(0xffffffffu, top > ref + 8.0f || vtop > vref)) {
            const float now = fmaxf(ref, top);
            const float f = ref == NINF ? 0.0f : ex2(ref - now);
            const float fo = f * ex2(vref - vtop);
            ref = now;
            vref = vtop;
            sum *= f;
            if (i > 0) {
              ok = wait(&odone[q], (g - 1) & 1, abort_flag);
              if (!ok) break;
              tc_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                tmem_ld32(o_at + c, s);
                wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) s[k] = __float_as_uint(__uint_as_float(s[k]) * fo);
                tmem_st32(o_at + c, s);
              }
              wait_st();
            }
          }
          const float base = (float)P_SHIFT - fmaxf(ref, -3.0e38f);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_ld32(s_at + 32 * c, s);
            wait_ld();
            const float f = fac * ex[c].x, shift = ex[c].y - vref, at = base + shift;
            float part = 0.0f;
#pragma unroll
            for (int k = 0; k < 32; ++k) s[k] = __float_as_uint(fmaf(__uint_as_float(s[k]), f, at));
            masked(c);
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const float a = ex2(__uint_as_float(s[k])), d = ex2(__uint_as_float(s[k + 1]));
              part += a + d;
              pk[k / 2] = pack_half(a, d);
            }
            sum = fmaf(part, ex2(-shift), sum);
            tmem_st16(s_at + 16 * c, pk);
          }
          // value scales that stand for NaN: their groups, in the rows that see the token
          const uint32_t* od = odds + (g & 3) * UNP * NG;
#pragma unroll 1
          for (int w = 0; w < UNP; ++w)
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
              const uint32_t bits = od[w * NG + gr];
              if (bits) {
                const int lo = min(max(seen.x - tok - 32 * w, 0), 32), hi = min(max(seen.y - tok - 32 * w, 0), 32);
                const uint32_t in = hi > lo ? (hi == 32 ? ~0u : (1u << hi) - 1) & ~((1u << lo) - 1) : 0u;
                if (bits & in) poison |= 1u << gr;
              }
            }
          wait_st();
          tc_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&pfull[q]);
        }
        // ---- O to shared memory (in K's and V's place, once no MMA reads them), row by row
        if (n > 0) {
          ok = ok && wait(&odone[q], (step + n - 1) & 1, abort_flag);
          if (tiles_q == 2) ok = ok && wait(&odone[q ^ 1], (step + n - 1) & 1, abort_flag);
          tc_after();
        }
        r_ml[rr] = make_float2(ref, sum * (1.0f / (1 << P_SHIFT)));
        const float back = ex2(vref - (float)P_SHIFT);
        float* o_row = reinterpret_cast<float*>(smem + L::O_K) + rr * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t s[32];
          if (n > 0 && ok) {
            tmem_ld32(o_at + c, s);
            wait_ld();
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) s[k] = 0;
          }
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            float x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              x[u] = __uint_as_float(s[k + u]) * back;
              // column jj 64 + r 8 + 2 i + hi is coordinate 32 (2 jj + hi) + 4 r + i
              if (poison >> (((c >> 6) * 2 + (u & 1)) / JG) & 1) x[u] = __int_as_float(0x7fffffff);
            }
            *reinterpret_cast<float4*>(o_row + ((((c + k) / 4) ^ (rr & (D / 4 - 1) & 31)) * 4)) = make_float4(x[0], x[1], x[2], x[3]);
          }
        }
        tc_before();
      }
    } else if (warp < SOFT + UNP) {
      // ======================= fetch and unpack: cache tile w of every step
      const int w = warp - SOFT, r = lane >> 2, c = lane & 3;
      const uint32_t raw = smem_u32(smem) + L::O_RAW + w * L::RAW;
      const uint32_t raw_v = raw + L::CODES, raw_s = raw + 2 * L::CODES;
      int64_t my_at = -1;
      auto at_of = [&](int i) -> int64_t {  // the tile of step i, or -1; lanes look 32 steps ahead
        return __shfl_sync(0xffffffffu, my_at, i & 31);
      };
      auto look = [&](int i) {
        if (i & 31) return;
        const int mine = i + lane, tok = tok_a + mine * TOK + 32 * w;
        my_at = -1;
        if (mine < n && tok < high) {
          my_at = kv4_tile_at(p.c, b, tok >> 5, h);
          if (my_at < 0) atomicExch(&g_kv4_rows_error, (int)ROT_EINVAL);
        }
      };
      auto load_k = [&](int i, int64_t at) {
        if (at >= 0 && lane == 0) {
          mbar_expect(&rawk[w], L::CODES + L::SCALES);
          bulk_load(raw, p.c.data + at, L::CODES, &rawk[w]);
          bulk_load(raw_s + (i & 1) * L::SCALES, p.c.data + at + 2 * L::CODES, L::SCALES, &rawk[w]);
        }
      };
      auto load_v = [&](int64_t at) {
        if (at >= 0 && lane == 0) {
          mbar_expect(&rawv[w], L::CODES);
          bulk_load(raw_v, p.c.data + at + L::CODES, L::CODES, &rawv[w]);
        }
      };
      look(0);
      int64_t at = n > 0 ? at_of(0) : -1;
      load_k(0, at);
      load_v(at);
      for (int i = 0; i < n && ok; ++i) {
        const uint32_t g = step + i, s = g & 1;
        const int tok = tok_a + i * TOK + 32 * w;
        int64_t next = -1;
        if (i + 1 < n) {
          look(i + 1);
          next = at_of(i + 1);
        }
        const bool here = at >= 0;
        const uint32_t sc = raw_s + (i & 1) * L::SCALES;
        // ---- exponents of the largest scales (tokens outside the sequence do not count)
        float kx = 1.0f, vx = -14.0f, kdown = 1.0f, vdown = 1.0f;
        if (here) {
          ok = wait(&rawk[w], got & 1, abort_flag);
          if (!ok) break;
          // this lane's token: its NG key scales, and by pairs (lane / 2) its value scales
          const bool in = tok + lane >= low && tok + lane < high;
          uint16_t vsc[NG];
          float kb = 0.0f, vb = 0.0f;
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            uint16_t a;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(a) : "r"(sc + (lane * NG + gr) * 2));
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(vsc[gr]) : "r"(sc + 64 * NG + ((lane >> 1) * NG + gr) * 4 + (lane & 1) * 2));
            if (in && (a & 0x7c00u) != 0x7c00u) kb = fmaxf(kb, __half2float(__ushort_as_half(a)));
            const bool odd = (vsc[gr] & 0x7c00u) == 0x7c00u;
            if (in && !odd) vb = fmaxf(vb, __half2float(__ushort_as_half(vsc[gr])));
            const uint32_t bits = __ballot_sync(0xffffffffu, in && odd);
            if (lane == 0) odds[((g & 3) * UNP + w) * NG + gr] = bits;
          }
#pragma unroll
          for (int x = 1; x < 32; x *= 2) {
            kb = fmaxf(kb, __shfl_xor_sync(0xffffffffu, kb, x));
            vb = fmaxf(vb, __shfl_xor_sync(0xffffffffu, vb, x));
          }
          const int ke = min(max((int)(__float_as_uint(kb) >> 23) - 126, -14), 16);  // kb <= 2^ke
          const int ve = min(max((int)(__float_as_uint(vb) >> 23) - 126, -14), 16);
          kx = __uint_as_float((uint32_t)(127 + ke) << 23);
          kdown = __uint_as_float((uint32_t)(127 - ke) << 23);
          vx = (float)ve;
          vdown = __uint_as_float((uint32_t)(127 - ve) << 23);
        } else if (lane < NG) {
          odds[((g & 3) * UNP + w) * NG + lane] = 0;
        }
        if (lane == 0) exps[(g & 3) * UNP + w] = make_float2(kx, vx);
        __syncwarp();
        if (lane == 0) mbar_arrive(&xfull[g & 3]);
        // ---- keys (tokens outside the sequence give logits that the softmax masks)
        ok = wait(&kempty[s], ((g >> 1) & 1) ^ 1, abort_flag);
        if (!ok) break;
        const uint32_t k_to = smem_u32(smem) + L::O_K + s * L::KV;
        const uint32_t kd = (uint32_t)__half_as_ushort(__float2half_rn(kdown)) * 0x00010001u;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int t = 8 * m + r, row = 32 * w + t;
          uint32_t word[J];
          if (here) lds<J>(raw + t * (D / 2) + c * (D / 8), word);
#pragma unroll
          for (int j = 0; j < J; ++j) {
            uint32_t v[4] = {0, 0, 0, 0};
            if (here) {
              uint16_t a;
              asm volatile("ld.shared.u16 %0, [%1];" : "=h"(a) : "r"(sc + (t * NG + j / JG) * 2));
              // an infinite scale (codes of 0) has to make the logit NaN: 0 * infinity does
              unpack(word[j], mul_half2((uint32_t)a * 0x00010001u, kd), v);
            }
            const int q8 = 4 * j + c;
            sts128(k_to + (q8 >> 3) * (TOK * 128) + row * 128 + (((q8 & 7) ^ (row & 7)) << 4), v);
          }
        }
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kfull[s]);
        load_k(i + 1, next);
        // ---- values (zeros outside the sequence and for scales that stand for NaN)
        if (here) ok = wait(&rawv[w], got & 1, abort_flag);
        ok = ok && wait(&vempty[s], ((g >> 1) & 1) ^ 1, abort_flag);
        if (!ok) break;
        const uint32_t v_to = smem_u32(smem) + L::O_V + s * L::KV;
        const uint32_t vd = (uint32_t)__half_as_ushort(__float2half_rn(vdown)) * 0x00010001u;
#pragma unroll
        for (int m = 0; m < 4; ++m) {  // eights of tokens: this lane's are 8 m + 2 c + b
          uint32_t word[J], scale[NG];  // words: blocks of b = 0, then of b = 1; scales: pairs (b = 0, b = 1)
          if (here) {
            lds<J>(raw_v + m * (4 * D) + (r * 4 + c) * (D / 8), word);
            lds<NG>(sc + 64 * NG + (4 * m + c) * (4 * NG), scale);
            const int t = tok + 8 * m + 2 * c;
            const uint32_t keep = (t >= low && t < high ? 0xffffu : 0u) | (t + 1 >= low && t + 1 < high ? 0xffff0000u : 0u);
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) scale[gr] = mul_half2(scale[gr] & keep & ~odd_halves(scale[gr]), vd);
          }
#pragma unroll
          for (int bb = 0; bb < 2; ++bb) {
            const int row = 32 * w + 8 * m + 2 * c + bb;
#pragma unroll
            for (int jj = 0; jj < J / 2; ++jj) {
              uint32_t v[4] = {0, 0, 0, 0};
              if (here) {
                // lower halves are block 2 jj, upper ones 2 jj + 1
                const uint32_t s2 = prmt(scale[2 * jj / JG], scale[(2 * jj + 1) / JG], bb ? 0x7632 : 0x5410);
                unpack(word[bb * (J / 2) + jj], s2, v);
              }
              sts128(v_to + jj * (TOK * 128) + row * 128 + ((r ^ (row & 7)) << 4), v);
            }
          }
        }
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&vfull[s]);
        load_v(next);
        got += here;
        at = next;
      }
      if (!ok) {  // copies that are still in flight get their time before the memory is given up
        const unsigned long long limit = WAIT_NS;
        unsigned long long t0, now;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
        do asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
        while (now - t0 < limit / 100);
      }
    } else {
      // ======================= MMA issue
      const uint32_t q_at = smem_u32(smem) + L::O_Q, k_at = smem_u32(smem) + L::O_K, v_at = smem_u32(smem) + L::O_V;
      auto pv = [&](int q, int i, bool last_q) {  // O += P V of step i
        const uint32_t g = step + i, s = g & 1;
        ok = ok && wait(&pfull[q], g & 1, abort_flag) && wait(&vfull[s], (g >> 1) & 1, abort_flag);
        if (!ok) return;
        tc_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < TOK / 16; ++k)
            mma_ts(tmem + 256 + q * D, tmem + q * 128 + 8 * k, desc(v_at + s * L::KV + k * 2048, TOK * 128, 1024), idesc(D, true),
                   i > 0 || k > 0);
          commit(&odone[q]);
          if (last_q) commit(&vempty[s]);
        }
        __syncwarp();
      };
      for (int i = 0; i < n && ok; ++i) {
        const uint32_t g = step + i, s = g & 1;
        ok = wait(&kfull[s], (g >> 1) & 1, abort_flag);
        for (int q = 0; q < tiles_q && ok; ++q) {
          if (i > 0) pv(q, i - 1, q == tiles_q - 1);
          if (!ok) break;
          tc_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ss(tmem + q * 128, desc(q_at + q * (128 * D * 2) + (k >> 2) * (128 * 128) + (k & 3) * 32, 16, 1024),
                     desc(k_at + s * L::KV + (k >> 2) * (TOK * 128) + (k & 3) * 32, 16, 1024), idesc(TOK, false), k > 0);
            commit(&sfull[q]);
            if (q == tiles_q - 1) commit(&kempty[s]);
          }
          __syncwarp();
        }
      }
      for (int q = 0; q < tiles_q && n > 0; ++q) pv(q, n - 1, q == tiles_q - 1);
      if (!ok) {  // MMAs that were issued end by themselves: give them a millisecond
        unsigned long long t0, now;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
        do asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
        while (now - t0 < 1000000ull);
      }
    }
    step += n;
    __syncthreads();
    ok = *abort_flag == 0;

    // ---- rows to their place, by whole warps
    for (int rr = warp; rr < tiles_q * 128; rr += WARPS) {
      const int row = row0 + rr;
      if (row >= n_rows) break;
      const float2 ml = r_ml[rr];
      const float* o_row = reinterpret_cast<const float*>(smem + L::O_K) + rr * D;
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int d = lane * V + i, col = (d >> 6) * 64 + ((d & 31) >> 2) * 8 + 2 * (d & 3) + ((d >> 5) & 1);
        o[i] = o_row[((col / 4) ^ (rr & (D / 4 - 1) & 31)) * 4 + (col & 3)];
      }
      const int64_t out_row = (first + row / p.share) * p.Hq + (int64_t)h * p.share + row % p.share;
      if (p.splits == 1) {
        finish_row<D>(p, o, ml.y, out_row, lane);
      } else {
        float* dst = p.part + (out_row * p.splits + split) * D + lane * V;
#pragma unroll
        for (int i = 0; i < V; ++i) dst[i] = o[i];
        if (lane == 0) {
          p.part_ml[(out_row * p.splits + split) * 2] = ml.x;
          p.part_ml[(out_row * p.splits + split) * 2 + 1] = ml.y;
        }
      }
    }
    __syncthreads();
    if (!ok) break;
  }
  tc_before();
  __syncthreads();
  if (warp == WARPS - 1) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

template <int D, int NG>
rot_status run(const Params& p, bool q_f32, cudaStream_t s) {
  const int64_t ctas = (int64_t)p.c.B * p.chunks * p.c.heads * p.splits;
  constexpr int smem = Lay<D, NG>::SMEM;
  return q_f32 ? launch<rows_kernel<D, NG, true>>(ctas, CTA, smem, s, p)
               : launch<rows_kernel<D, NG, false>>(ctas, CTA, smem, s, p);
}

}  // namespace

rot_status kv4_rows_launch(const kv4::Params& p, int D, int NG, bool q_f32, cudaStream_t s) {
  switch (D * 16 + NG) {
    case 64 * 16 + 2: return run<64, 2>(p, q_f32, s);
    case 64 * 16 + 1: return run<64, 1>(p, q_f32, s);
    case 128 * 16 + 4: return run<128, 4>(p, q_f32, s);
    case 128 * 16 + 2: return run<128, 2>(p, q_f32, s);
    case 128 * 16 + 1: return run<128, 1>(p, q_f32, s);
    default: return set_error(ROT_EUNSUPPORTED, "kv4_attention: no kernel for many rows of this D and G");
  }
}

rot_status kv4_rows_fetch_device_error() {
  int v = 0;
  ROT_CUDA_TRY(cudaMemcpyFromSymbol(&v, g_kv4_rows_error, sizeof(int)));
  if (v) {
    int z = 0;
    ROT_CUDA_TRY(cudaMemcpyToSymbol(g_kv4_rows_error, &z, sizeof(int)));
    return set_error((rot_status)v, v == ROT_ETIMEOUT ? "a bounded wait in kv4_attention gave up"
                                                      : "kv4_attention: a page table named no page of the cache for a token");
  }
  return ROT_OK;
}

}  // namespace rotb
