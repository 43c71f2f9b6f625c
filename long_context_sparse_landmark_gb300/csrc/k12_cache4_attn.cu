// K12: attention of a few query tokens over the 4-bit KV cache, in full or over a
// window.
//
// Mathematics, per query row, in log2 units: s_j = scale log2e <q, k_j>, out =
// sum_j 2^{s_j} v_j / sum_j 2^{s_j}.  A slot's codes times their scales over the
// slot's own largest, 2^x, are halves (code * 2^{13 - delta}, exact for a delta
// of up to 27; 0 beyond): k_j = 2^{x_j - 13} kh_j, and likewise v_j = 2^{y_j} vh_j.
// x goes into the score, y into the exponent of the weight that meets vh: w_j =
// 2^{(s_j - M) + (y_j - D)}.  M, to 2^60, is the largest s so far, the
// denominator's reference, and M + D, to 2^1.5, the largest s + y, the output's;
// D is kept as an offset of M, so that a large score does not round the value
// scale away.  No slot's scales touch another's (the slow path: read_scales, softmax).
//
// Slots' scales hardly differ by more than a few binades.  So a warp holds one
// reference for K's scales and one for V's, 2^{rk} and 2^{rv}: where none of a
// pair's scales is above its reference or more than 27 binades (V: 12) below, code *
// 2^{13 - (r - x)} is a half, exactly, all scores have one factor and all values one
// unit, and an exponent is one multiply-add of a raw score (fits, softmax_one).  V's
// limit is that of the weights' halves: in one unit a weight has no part of its
// value's scale, and one so small that its half is subnormal is off by 2^-34 of the
// row's largest, times values 2^12 times the largest's at most.  Where a
// pair does not fit, new references are tried, with 4 binades of room; where those do
// not either, each slot's own scales are taken.
//
// The work is read once, 136 bytes a slot and KV head of 128 dims, shared by the
// group's rows: half of what the 8-bit cache takes.  Instructions bound it almost as
// much as HBM does: 24 sequences of 16K to 32K slots, 64 heads on 8, run at 71 % of
// DRAM's peak with 58 % of the issue slots, 45 % of the integer pipe (where codes
// become halves, at half its rate) and 30 % of the tensor pipe in use, about 500
// instructions a chunk of 32 slots; 64 such sequences take 285 us, 6.15 TB/s, where
// each slot's own scales took 371.  The list of 32-slot chunks, its cut and the join
// are the 8-bit cache's (cache_attn.cuh).
//
// All rows run on the tensor cores (mma.sync, fp16 operands): keys are the MMA's
// 16 rows and query rows its 8 columns, so that a group of 8 heads wastes nothing.
// (tcgen05, with slots as its 128 rows and query rows as its columns, wants the codes
// widened in shared memory, 64 KB written and read again for every 128 slots; the
// tensor pipe is not what bounds this.  Measured with S and O in tensor memory and two
// CTAs an SM: 857 us for 419, 64 sequences of 16K to 32K slots, two tokens, 64 heads on
// 8; 94 for 52, 16 sequences, four tokens, a window of 4096.)
// A lane's share of a slot is a run of d / 4 dims of K, d / 8 of V: each within one
// scale, so a fragment takes a conversion of two codes and one multiplication.
// fp32 rows are two halves each, their weights too: 22 bits.
#include "cache4.cuh"
#include "cache_attn.cuh"

namespace msa {
namespace {

// Room above the largest weight when a reference is set from values in one unit, so
// that few chunks move it again: a move scales all of a warp's sums, and of 32 rows
// some row's maximum rises in most of a short range's chunks.  A weight's half keeps
// its 11 bits down to 2^-23 of the largest.  (Slots far apart have no room to spare.)
constexpr float kRoom = 5.f;
constexpr uint32_t kKSpan = 27, kVSpan = 12;  // binades of scales below a reference
constexpr float kTop = 13.f;  // a code of the slot's largest scale is code * 2^13

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&a),
                            *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&x);
}
// Reads of shared memory at an address and a constant: one instruction each, the
// lane's part of an address held over the chunks.
template <int kAt>
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4 + %5];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a), "n"(kAt));
  return v;
}
template <int kAt>
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2 + %3];" : "=r"(v.x), "=r"(v.y) : "r"(a), "n"(kAt));
  return v;
}
template <int kAt>
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1 + %2];" : "=r"(v) : "r"(a), "n"(kAt));
  return v;
}
template <int kAt>
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1 + %2];" : "=r"(v) : "r"(a), "n"(kAt));
  return v;
}
// f(0), f(1), ... f(kN - 1), each with a constant.
template <int kI>
struct Const {
  static constexpr int value = kI;
};
template <int kN, int kI = 0, typename F>
__device__ __forceinline__ void each(F f) {
  if constexpr (kI < kN) {
    f(Const<kI>{});
    each<kN, kI + 1>(f);
  }
}
// Bits of m from a, the others from b: one instruction, which the compiler does
// not find behind a shift.
__device__ __forceinline__ uint32_t select_bits(uint32_t m, uint32_t a, uint32_t b) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xca;" : "=r"(r) : "r"(m), "r"(a), "r"(b));
  return r;
}

// Scales of a slot (bytes of w) as halves 2^{13 - delta} below the largest, which
// is returned: groups 0 and 2 in h[0], 1 and 3 in h[1].
__device__ __forceinline__ uint32_t slot_scales(uint32_t w, uint32_t* h) {
  const uint32_t a = w & 0x00ff00ffu, b = (w >> 8) & 0x00ff00ffu;
  uint32_t m = __vmaxu2(a, b);
  m = max(m >> 16, m & 0xffffu);
  // (13 + 15) - delta as exponents of halves, 0 at the least: a half of 0.
  const uint32_t off = __byte_perm(28u - m, 0, 0x1010);
  h[0] = __viaddmax_s16x2(a, off, 0u) << 10;
  h[1] = __viaddmax_s16x2(b, off, 0u) << 10;
  return m;
}

// Of 8 kNt query rows, each kTerms halves.  kChunks: chunks that a warp takes together,
// two where the registers allow it and there are many (cache4_attn_pairs), so that
// one's fixed latencies pass in the other's shadow.
template <int D, int kNt, int kTerms, int kChunks = 1>
struct Body4 {
  static constexpr int kTile = 8 * kNt;
  static constexpr int kPerSm = kNt == 1 || kNt * kTerms == 2 ? 3 : 2;
  // CTAs an SM: 3 where 168 registers do (4 and 5 of 8 rows spill: 377 and 431 us for
  // 367, 64 sequences of 16K to 32K slots with each slot's own scales).
  static constexpr int kPair = kChunks;
  // Pairs under way.  16 bf16 rows, at 3 CTAs an SM, need no more than two (64
  // sequences of 16K to 32K slots, two tokens: 417 us with 2, 427 with 3; with 4 only 2
  // CTAs fit, 97 us for 68 with 8 sequences).
  static constexpr int kStages =
      (kPair == 2 || kNt == 4 ? 4 : kNt == 2 && kTerms == 1 ? 2 : 3) / kPair *
      (D == 128 ? 1 : 2);
  static constexpr bool kQShared = kNt > 1;
  static constexpr int kCodes = kChunk * D / 2, kScales = kChunk * D / kGroup4;  // of K, or of V
  static constexpr int kChunkBytes = 2 * kCodes + 2 * kScales;
  static constexpr int kStageBytes = kPair * kChunkBytes;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kKs = D / 16;  // k-steps over d
  static constexpr int kMt = D / 16;  // 16-row tiles of O^T
  static constexpr int kGroups = D / kGroup4;
  static constexpr int kUnset = -1000;

  // What a warp makes of a chunk's scales.
  struct Scales {
    float2 slot[kChunk];              // 2^x, and y
    uint32_t k[kChunk * kGroups];     // half 2^{13 - delta}, twice: [slot][group]
    uint16_t v[kGroups][40];          // the half: [group][slot], rows 80 bytes apart
    float refs[kNt >= 2 ? 4 * kNt * 32 : 4];  // see M() below
  };
  // Rows of a unit, for all warps: their fragments [term][k-step][tile][lane],
  // score scales and positions.
  struct Rows {
    uint2 q[kTerms][kKs * kNt * 32];
    float scale[kTile];
    int pos[kTile];
  };
  static constexpr int kSmem = kWarps * (kRingBytes + static_cast<int>(sizeof(Scales))) +
                               static_cast<int>(sizeof(Rows));
  static_assert(kWarps * kRingBytes >= kWarps * kTile * (D + 4) * 4, "sums must fit the rings");
  static_assert(sizeof(Scales) % 16 == 0 && kStageBytes % 16 == 0, "16-byte pieces");

  uint32_t q[kTerms][kQShared ? 1 : kKs][kQShared ? 1 : kNt][2];
  float o[kMt][kNt][4];
  float l[kNt][2];  // in units of 2^M, o of 2^{M + D0 - kPBits}
  // M and D0 of rows 2t, 2t+1: looked at where a reference moves or a chunk does not
  // fit.  Those of two and four tiles are in shared memory: with 32 rows in registers
  // 304 bytes spilled (162 still do at d = 128, 255 registers), and 16 rows are 3 CTAs
  // an SM (168 registers, 28 bytes spilled) without them.
  static constexpr bool kCold = kNt >= 2;
  struct Refs {
    float v[2][kNt][2];
  } refs;
  float* cold;
  __device__ __forceinline__ float M(int n, int r) const {
    return kCold ? cold[(2 * n + r) * 32] : refs.v[0][n][r];
  }
  __device__ __forceinline__ float D0(int n, int r) const {
    return kCold ? cold[(2 * kNt + 2 * n + r) * 32] : refs.v[1][n][r];
  }
  __device__ __forceinline__ void set(int n, int r, float m, float d) {
    if (kCold) {
      cold[(2 * n + r) * 32] = m;
      cold[(2 * kNt + 2 * n + r) * 32] = d;
    } else {
      refs.v[0][n][r] = m;
      refs.v[1][n][r] = d;
    }
  }
  // Score scale (log2 units).
  __device__ __forceinline__ float qs(int n, int r) const {
    return rows->scale[8 * n + 2 * (threadIdx.x & 3) + r];
  }

  __device__ __forceinline__ static Rows& rows_of(uint8_t* smem) {
    return *reinterpret_cast<Rows*>(smem +
                                    kWarps * (kRingBytes + static_cast<int>(sizeof(Scales))));
  }

  // The CTA writes them: a thread takes 8 values of a row.
  __device__ __forceinline__ static void load_rows(const CacheAttnArgs& a, const Plan& p,
                                                   const Entry& e, int c, int rt, uint8_t* smem) {
    constexpr int kP = D / 8, kOwn = D / 32;  // pieces of a row, and of a lane
    Rows& rows = rows_of(smem);
#pragma unroll 1
    for (int i = threadIdx.x; i < kTile * kP; i += kThreads) {  // whole warps
      const int r = i / kP, pc = i - r * kP, m = rt * kTile + r;
      int t, h;
      row_of(a, e, c, min(m, p.rows - 1), &t, &h);
      const int64_t at = ((static_cast<int64_t>(e.b) * a.T + t) * a.Hq + h) * D + 8 * pc;
      float v[8], mx = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = 0.f;
      if (m < p.rows && MSA_IN_RANGE(at, 8, static_cast<int64_t>(a.s.batch) * a.T * a.Hq * D,
                                     a.status)) {
        if constexpr (kTerms == 1) {
          const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[2 * k] = __uint_as_float(w[k] << 16);
            v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
          }
        } else {
          const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at);
          const float4 x = s[0], y = s[1];
          v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
          v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(v[k]));
#pragma unroll
      for (int o2 = 1; o2 < kP; o2 <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o2));
      // 2^k brings the row's largest magnitude to [2^14, 2^15).
      int k2 = mx > 0.f ? 14 + 127 - static_cast<int>(__float_as_uint(mx) >> 23) : 0;
      k2 = k2 > 100 ? 100 : k2;
      const float up = pow2i(k2);
      // Lane t4's dims of k-step ks are (D / 4) t4 + 4 ks + 0..3.
      const int ks = 2 * (pc % kOwn);
      const int lane = (r & 7) * 4 + pc / kOwn;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= up;
#pragma unroll
      for (int term = 0; term < kTerms; ++term) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __half2 x = __floats2half2_rn(v[2 * k], v[2 * k + 1]);
          w[k] = *reinterpret_cast<const uint32_t*>(&x);
          if (term + 1 < kTerms) {  // what the half leaves, exactly
            const float2 f = __half22float2(x);
            v[2 * k] -= f.x;
            v[2 * k + 1] -= f.y;
          }
        }
        uint2* to = rows.q[term] + (ks * kNt + (r >> 3)) * 32 + lane;
        to[0] = make_uint2(w[0], w[1]);
        to[kNt * 32] = make_uint2(w[2], w[3]);
      }
      if (pc == 0) {
        rows.scale[r] = a.scale * kLog2e * pow2i(-k2) * 0x1p-13f;
        rows.pos[r] = e.len - a.T + t;
      }
    }
  }

  // What the scales are taken over by a chunk that fits (see fits()): bytes of K
  // and V, or kUnset; and what follows from them and the references above.
  int rk, rv;
  float2 f[kNt];     // of a raw score, to log2 units
  float2 base[kNt];  // added to a score: the exponent of its weight
  float2 back[kNt];  // of a weight, to units of 2^M
  float lvs;         // log2 of V's unit
  bool level;        // a weight tells the denominator's term in every row

  // The lane's parts of the addresses below, from a stage's start.
  uint32_t at_k, at_v[2], at_ks, at_vs;

  const Rows* rows;
  Scales* scales;

  __device__ __forceinline__ void begin(uint8_t* smem) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    rows = &rows_of(smem);
    // Slots g (+ 8, + 16 st) of K: words t4's; slots 2 t4 + q (+ 8, + 16 st) of V: g's.
    at_k = D == 128 ? k_at(g, t4) : k_at(g, t4 >> 1) + 8 * (t4 & 1);
#pragma unroll
    for (int q2 = 0; q2 < 2; ++q2)
      at_v[q2] = D == 128 ? v_at(2 * t4 + q2, g >> 1) + 8 * (g & 1)
                          : v_at(2 * t4 + q2, g >> 2) + 4 * (g & 3);
    at_ks = 2 * kCodes + g * kGroups + (D == 128 ? t4 : t4 >> 1);
    at_vs = 2 * kCodes + kScales + 2 * t4 * kGroups + (D == 128 ? g >> 1 : g >> 2);
    scales = reinterpret_cast<Scales*>(smem + kWarps * kRingBytes) + (threadIdx.x >> 5);
    cold = scales->refs + lane;
    rk = rv = kUnset;
    level = false;
#pragma unroll
    for (int n = 0; n < kNt; ++n) {
      if constexpr (!kQShared) {
#pragma unroll
        for (int term = 0; term < kTerms; ++term)
#pragma unroll
          for (int ks = 0; ks < kKs; ++ks) {
            const uint2 x = rows->q[term][(ks * kNt + n) * 32 + lane];
            q[term][ks][n][0] = x.x;
            q[term][ks][n][1] = x.y;
          }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        set(n, r, -INFINITY, 0.f);
        l[n][r] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kMt; ++i)
#pragma unroll
      for (int n = 0; n < kNt; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][n][k] = 0.f;
  }

  // A warp's chunks pass through a ring of its own: K codes [32][D / 2], V codes
  // likewise with rows and 16-byte pieces moved about so that the fragment reads
  // below meet no bank twice, then the scales.
  __device__ __forceinline__ static int k_at(int row, int piece) {
    return row * (D / 2) + (piece << 4);
  }
  __device__ __forceinline__ static int v_at(int row, int piece) {
    return kCodes + (D == 128 ? (row ^ ((row >> 1) & 1)) * 64 + ((piece ^ ((row >> 1) & 2)) << 4)
                              : (row ^ ((row >> 2) & 1)) * 32 + (piece << 4));
  }
  // Starts the copy of chunk `x` of the pool (32 slots of a page and head) to `to`,
  // the lane's place in a stage; k, v, e: the lane's place in chunk 0 of the codes
  // and of K's or V's scales.
  struct Place {
    const uint8_t *k, *v, *e;
    uint32_t to_v;  // of V's pieces, from `to`
  };
  __device__ __forceinline__ static Place place(const Cache4AttnArgs& a) {
    constexpr int kSp = kScales / 16;  // pieces of K's scales, and of V's
    const int lane = threadIdx.x & 31;
    Place p;
    p.k = a.c.k_codes + lane * 16;
    p.v = a.c.v_codes + lane * 16;
    p.e = (lane < kSp ? a.k_exp : a.v_exp) + (lane % kSp) * 16;
    p.to_v = v_at(lane / (D / 32), lane % (D / 32)) - lane * 16;
    return p;
  }
  __device__ __forceinline__ static void copy(const Cache4AttnArgs& a, const Place& p, uint32_t x,
                                              uint32_t to) {
    static_assert(32 * 16 % (8 * D / 2) == 0, "a warp's pieces: rows whose places are alike");
    if (!MSA_IN_RANGE(static_cast<int64_t>(x) * kChunk, kChunk,
                      a.c.n_pages * a.c.Hkv * a.c.block, a.status))
      return;
    const uint8_t* k = p.k + static_cast<uint64_t>(x) * kCodes;
    const uint8_t* v = p.v + static_cast<uint64_t>(x) * kCodes;
    each<kCodes / 512>([&](auto i) {
      asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %2], 16;" ::"r"(to), "l"(k),
                   "n"(decltype(i)::value * 512)
                   : "memory");
    });
    each<kCodes / 512>([&](auto i) {
      asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %2], 16;" ::"r"(to + p.to_v),
                   "l"(v), "n"(decltype(i)::value * 512)
                   : "memory");
    });
    if ((threadIdx.x & 31) < 2 * (kScales / 16))
      asm volatile("cp.async.cg.shared.global [%0 + %2], [%1], 16;" ::"r"(to),
                   "l"(p.e + static_cast<uint64_t>(x) * kScales), "n"(2 * kCodes)
                   : "memory");
  }

  // Whether no scale of the pair is above the warp's references or further below than
  // their spans: then code * 2^{13 - (r - x)} are halves, exactly, and the slots' own
  // scales need no looking at.  (Slots that no row attends: see blank().)
  __device__ __forceinline__ bool fits(uint32_t stage) const {
    const uint32_t at = stage + (threadIdx.x & 31) * kGroups;
    const uint32_t k2 = __byte_perm(rk, 0, 0x1010), v2 = __byte_perm(rv, 0, 0x1010);
    uint32_t mk = 0, mv = 0;
    each<kPair>([&](auto c) {
      constexpr int k_from = decltype(c)::value * kChunkBytes + 2 * kCodes, v_from = k_from + kScales;
      if constexpr (D == 128) {
        const uint32_t kw = lds32<k_from>(at), vw = lds32<v_from>(at);
        mk = __vimax3_u16x2(mk, k2 - __byte_perm(kw, 0, 0x4240), k2 - __byte_perm(kw, 0, 0x4341));
        mv = __vimax3_u16x2(mv, v2 - __byte_perm(vw, 0, 0x4240), v2 - __byte_perm(vw, 0, 0x4341));
      } else {
        const uint32_t k0 = lds8<k_from>(at), k1 = lds8<k_from + 1>(at);
        const uint32_t v0 = lds8<v_from>(at), v1 = lds8<v_from + 1>(at);
        mk = __vmaxu2(mk, k2 - (k0 | k1 << 16));
        mv = __vmaxu2(mv, v2 - (v0 | v1 << 16));
      }
    });
    // (A byte above its reference leaves a borrow, and 0xff.. in its own half.)
    constexpr uint32_t kK = kKSpan * 0x10001u, kV = kVSpan * 0x10001u;
    return __all_sync(0xffffffffu, __vmaxu2(mk, kK) == kK && __vmaxu2(mv, kV) == kV);
  }
  // Slots that no row attends hold anything: their scales become the references,
  // so that they fit and are finite.  `off`: bit c for the lane's slot of chunk c.
  __device__ __forceinline__ void blank(uint32_t stage, uint32_t off) const {
    const uint32_t at = stage + (threadIdx.x & 31) * kGroups;
    const uint32_t k = rk == kUnset ? 0x01010101u : rk * 0x01010101u;
    const uint32_t v = rv == kUnset ? 0x01010101u : rv * 0x01010101u;
    each<kPair>([&](auto c) {
      constexpr int from = decltype(c)::value * kChunkBytes + 2 * kCodes;
      if (off >> decltype(c)::value & 1) {
        if constexpr (D == 128) {
          asm volatile("st.shared.u32 [%0 + %1], %2;" ::"r"(at), "n"(from), "r"(k) : "memory");
          asm volatile("st.shared.u32 [%0 + %1], %2;" ::"r"(at), "n"(from + kScales), "r"(v)
                       : "memory");
        } else {
          asm volatile("st.shared.u16 [%0 + %1], %2;" ::"r"(at), "n"(from),
                       "h"(static_cast<uint16_t>(k))
                       : "memory");
          asm volatile("st.shared.u16 [%0 + %1], %2;" ::"r"(at), "n"(from + kScales),
                       "h"(static_cast<uint16_t>(v))
                       : "memory");
        }
      }
    });
    __syncwarp();
  }
  // References for a pair that does not fit, with some room above its largest
  // scales; false if there are none.
  __device__ __forceinline__ bool refer(uint32_t stage, uint32_t off) {
    const uint32_t at = stage + (threadIdx.x & 31) * kGroups;
    uint32_t k = 1, v = 1;
    each<kPair * kGroups>([&](auto i) {
      constexpr int c = decltype(i)::value / kGroups, j = decltype(i)::value % kGroups;
      const uint32_t kb = lds8<c * kChunkBytes + 2 * kCodes + j>(at);
      const uint32_t vb = lds8<c * kChunkBytes + 2 * kCodes + kScales + j>(at);
      if (!(off >> c & 1)) {
        k = max(k, kb);
        v = max(v, vb);
      }
    });
    k = __reduce_max_sync(0xffffffffu, k);
    v = __reduce_max_sync(0xffffffffu, v);
    if (k == 255 || v == 255) return false;
    const int k0 = rk, v0 = rv;
    rk = min(static_cast<int>(k) + 4, 254);  // below NaN's, which never fits
    rv = min(static_cast<int>(v) + 4, 254);
    if (__any_sync(0xffffffffu, off)) blank(stage, off);
    if (!fits(stage)) {
      rk = k0;
      rv = v0;
      return false;
    }
    follow();
    return true;
  }
  // What follows from the references.
  __device__ __forceinline__ void follow() {
    if (rk == kUnset) return;
    // 2^{rk - 127} may pass a float's range by the room above: two factors.
    const float k = pow2i(rk - 131);
    lvs = static_cast<float>(rv) - 127.f - kTop;
    bool in = true;
#pragma unroll
    for (int n = 0; n < kNt; ++n) {
      f[n] = make_float2(qs(n, 0) * 16.f * k, qs(n, 1) * 16.f * k);
      const float2 up = make_float2(kPBits + (lvs - D0(n, 0)), kPBits + (lvs - D0(n, 1)));
      base[n] = make_float2(up.x - M(n, 0), up.y - M(n, 1));
      back[n] = make_float2(ex2(-up.x), ex2(-up.y));
      // No slot yet: the first score moves the references.
#pragma unroll
      for (int r = 0; r < 2; ++r)
        in &= M(n, r) == -INFINITY || lvs - D0(n, r) >= -40.f;
    }
    level = __all_sync(0xffffffffu, in);
  }

  // A lane a slot: its scales.
  __device__ __forceinline__ void read_scales(uint32_t stage) {
    const int lane = threadIdx.x & 31;
    const uint32_t at = stage + lane * kGroups;
    uint32_t kw, vw;
    if constexpr (D == 128) {
      kw = lds32<2 * kCodes>(at);
      vw = lds32<2 * kCodes + kScales>(at);
    } else {
      kw = lds8<2 * kCodes>(at) | lds8<2 * kCodes + 1>(at) << 8;
      vw = lds8<2 * kCodes + kScales>(at) | lds8<2 * kCodes + kScales + 1>(at) << 8;
    }
    uint32_t kh[2], vh[2];
    const uint32_t x = slot_scales(kw, kh), y = slot_scales(vw, vh);
    const float ks = e8m0_to_float(x);
    const float lvs = y == 255 ? __uint_as_float(0x7fc00000u) : static_cast<float>(y) - 127.f - kTop;
    scales->slot[lane] = make_float2(ks, lvs);
    if constexpr (D == 128) {
      reinterpret_cast<uint4*>(scales->k)[lane] =
          make_uint4(__byte_perm(kh[0], 0, 0x1010), __byte_perm(kh[1], 0, 0x1010),
                     __byte_perm(kh[0], 0, 0x3232), __byte_perm(kh[1], 0, 0x3232));
      scales->v[2][lane] = static_cast<uint16_t>(vh[0] >> 16);
      scales->v[3][lane] = static_cast<uint16_t>(vh[1] >> 16);
    } else {
      reinterpret_cast<uint2*>(scales->k)[lane] =
          make_uint2(__byte_perm(kh[0], 0, 0x1010), __byte_perm(kh[1], 0, 0x1010));
    }
    scales->v[0][lane] = static_cast<uint16_t>(vh[0]);
    scales->v[1][lane] = static_cast<uint16_t>(vh[1]);
  }

  float s[2 * kPair][kNt][4];  // [16-slot step][tile][slot g, row 2t, 2t+1; slot g + 8, ...]

  // Raw scores of the chunk at `stage`, the kC-th of a pair.
  template <bool kOwn, int kC>
  __device__ __forceinline__ void scores(uint32_t stage) {
    constexpr int kW = D / 32;  // words of a K row a lane holds, 8 dims each
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int st = 0; st < 2; ++st)
#pragma unroll
      for (int n = 0; n < kNt; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[2 * kC + st][n][k] = 0.f;
    uint32_t kw[2][2][kW], sc[2][2];
    const uint32_t from = stage + at_k, from_s = stage + at_ks;
    each<4>([&](auto i) {
      constexpr int st = decltype(i)::value >> 1, r = decltype(i)::value & 1;
      constexpr int row = 16 * st + 8 * r;
      if constexpr (kOwn)
        sc[st][r] = scales->k[(row + g) * kGroups + (D == 128 ? t4 : t4 >> 1)];
      else  // 28 - (rk - x) as the exponent of a half, twice
        sc[st][r] = lds8<row * kGroups>(from_s) * 0x04000400u + (28u - rk) * 0x04000400u;
      if constexpr (D == 128) {
        const uint4 w = lds128<row * (D / 2)>(from);
        kw[st][r][0] = w.x, kw[st][r][1] = w.y, kw[st][r][2] = w.z, kw[st][r][3] = w.w;
      } else {
        const uint2 w = lds64<row * (D / 2)>(from);
        kw[st][r][0] = w.x, kw[st][r][1] = w.y;
      }
    });
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      uint32_t x[2][2][4];
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          e2m1x8_to_half2(kw[st][r][w], x[st][r]);
#pragma unroll
          for (int k = 0; k < 4; ++k) x[st][r][k] = hmul2(x[st][r][k], sc[st][r]);
        }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int term = kTerms - 1; term >= 0; --term)  // the smaller products first
#pragma unroll
          for (int n = 0; n < kNt; ++n) {
            const int ks = 2 * w + h;
            uint32_t b0, b1;
            if constexpr (kQShared) {
              const uint2 y = rows->q[term][(ks * kNt + n) * 32 + lane];
              b0 = y.x, b1 = y.y;
            } else {
              b0 = q[term][ks][n][0], b1 = q[term][ks][n][1];
            }
#pragma unroll
            for (int st = 0; st < 2; ++st) {
              const uint32_t fa[4] = {x[st][0][2 * h], x[st][1][2 * h], x[st][0][2 * h + 1],
                                      x[st][1][2 * h + 1]};
              mma16816(s[2 * kC + st][n], fa, b0, b1);
            }
          }
    }
  }

  // Softmax of the chunk's scores into halves pf[term][step][tile][b0, b1], and
  // the running sums.  kEdge: some slot is masked for some row.
  uint32_t pf[kTerms][2 * kPair][kNt][2];

  // The warp's largest of a row's value.
  __device__ __forceinline__ static float row_max(float x) {
#pragma unroll
    for (int o2 = 4; o2 < 32; o2 <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o2));
    return x;
  }
  // Moves a row's references: `top` its largest score, `to` that or M, `v` the
  // largest s + y, from `to`; room: above it.
  __device__ __forceinline__ void move(int n, int r, float top, float to, float v, float room) {
    const float up = top - M(n, r), kept = D0(n, r) - (to - M(n, r));
    if (v - kept > 0.f || up > 60.f) {
      const float off = fmaxf(kept, v + room);  // kept: the output's unit stays
      const float down = ex2(kept - off);
      l[n][r] *= ex2(M(n, r) - to);
#pragma unroll
      for (int i = 0; i < kMt; ++i) {
        o[i][n][r] *= down;
        o[i][n][2 + r] *= down;
      }
      set(n, r, to, off);
    }
  }

  __device__ __forceinline__ void put_weights(int st, int n, int k, float2 w) {
#pragma unroll
    for (int term = 0; term < kTerms; ++term) {
      const __half2 h = __floats2half2_rn(w.x, w.y);
      pf[term][st][n][k] = transpose8x8(*reinterpret_cast<const uint32_t*>(&h));
      if (term + 1 < kTerms) {
        const float2 x = __half22float2(h);
        w.x -= x.x;
        w.y -= x.y;
      }
    }
  }

  // Of a pair that fits: its scores are raw, its values in one unit.
  // kEdge: some slot is masked for some row; live: bit c for chunk c.
  template <bool kEdge>
  __device__ __forceinline__ void softmax_one(const CacheAttnArgs& a, int key0, uint32_t live) {
    if constexpr (kEdge) {
      const int g = (threadIdx.x & 31) >> 2, t4 = threadIdx.x & 3;
#pragma unroll
      for (int n = 0; n < kNt; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int p = rows->pos[8 * n + 2 * t4 + r];
#pragma unroll
          for (int st = 0; st < 2 * kPair; ++st)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int key = key0 + 16 * st + 8 * k + g;
              if (!(live >> (st >> 1) & 1) || key > p || p - key >= a.window)
                s[st][n][2 * k + r] = -INFINITY;
            }
        }
    }
    constexpr bool kKeep = kNt < 2;  // else they are computed twice: registers
    float2 z[2 * kPair][kKeep ? kNt : 1][2];
    const auto exponents = [&] {
      bool high = false;
#pragma unroll
      for (int n = 0; n < kNt; ++n) {
        float most[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int st = 0; st < 2 * kPair; ++st)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 y = make_float2(s[st][n][2 * k], s[st][n][2 * k + 1]);
            const float2 x = __ffma2_rn(y, f[n], base[n]);
            if constexpr (kKeep) z[st][n][k] = x;
            most[0] = fmaxf(most[0], x.x);
            most[1] = fmaxf(most[1], x.y);
          }
        high |= fmaxf(most[0], most[1]) > kPBits + 1.5f;
      }
      return high;
    };
    if (__any_sync(0xffffffffu, exponents())) {
#pragma unroll
      for (int n = 0; n < kNt; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float mx = -INFINITY;
#pragma unroll
          for (int st = 0; st < 2 * kPair; ++st)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              mx = fmaxf(mx, s[st][n][2 * k + r] * (r ? f[n].y : f[n].x));
          const float top = row_max(mx), to = fmaxf(M(n, r), top);
          move(n, r, top, to, (top - to) + lvs, kRoom);
        }
      follow();
      exponents();
    }
#pragma unroll
    for (int n = 0; n < kNt; ++n) {
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int st = 0; st < 2 * kPair; ++st)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 x =
              kKeep ? z[st][kKeep ? n : 0][k]
                    : __ffma2_rn(make_float2(s[st][n][2 * k], s[st][n][2 * k + 1]), f[n], base[n]);
          float2 w = make_float2(ex2(x.x), ex2(x.y));
          if (kEdge) {  // also where no slot was attended yet
            if (s[st][n][2 * k] == -INFINITY) w.x = 0.f;
            if (s[st][n][2 * k + 1] == -INFINITY) w.y = 0.f;
          }
          sum = __fadd2_rn(sum, w);
          put_weights(st, n, k, w);
        }
      const float2 d = __ffma2_rn(sum, back[n], make_float2(l[n][0], l[n][1]));
      l[n][0] = d.x;
      l[n][1] = d.y;
    }
  }

  // Of a chunk with its slots' own scales; masks are applied everywhere.  on: the
  // chunk has a page.
  __device__ __forceinline__ void softmax(const CacheAttnArgs& a, int key0, bool on) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    float2 lvs[2][2];  // [step][slot g, g + 8]
    float mx[kNt][2];
#pragma unroll
    for (int n = 0; n < kNt; ++n) mx[n][0] = mx[n][1] = -INFINITY;
#pragma unroll
    for (int st = 0; st < 2; ++st)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 of = scales->slot[16 * st + 8 * k + g];
        lvs[st][k] = make_float2(of.y, of.y);
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
          const float2 f = __fmul2_rn(make_float2(qs(n, 0), qs(n, 1)), make_float2(of.x, of.x));
          float2 y = __fmul2_rn(make_float2(s[st][n][2 * k], s[st][n][2 * k + 1]), f);
          const int key = key0 + 16 * st + 8 * k + g;
          const int p0 = rows->pos[8 * n + 2 * t4], p1 = rows->pos[8 * n + 2 * t4 + 1];
          if (!on || key > p0 || p0 - key >= a.window) y.x = -INFINITY;
          if (!on || key > p1 || p1 - key >= a.window) y.y = -INFINITY;
          s[st][n][2 * k] = y.x;
          s[st][n][2 * k + 1] = y.y;
          mx[n][0] = fmaxf(mx[n][0], y.x);
          mx[n][1] = fmaxf(mx[n][1], y.y);
        }
      }
    // A weight may exceed 2^14 by a factor 2^1.5 (the half's range allows it) and a
    // term of the denominator 1 by 2^60 before the references move, so that most
    // chunks move neither them nor the sums, and the lanes need not agree.
    float2 z[2][kNt][2];  // exponents of the weights
    const auto exponents = [&] {
      bool high = false;
#pragma unroll
      for (int n = 0; n < kNt; ++n) {
        const float2 minus_M = make_float2(-M(n, 0), -M(n, 1));
        const float2 base = make_float2(kPBits - D0(n, 0), kPBits - D0(n, 1));
        float most[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 t =
                __fadd2_rn(make_float2(s[st][n][2 * k], s[st][n][2 * k + 1]), minus_M);
            z[st][n][k] = __fadd2_rn(t, __fadd2_rn(lvs[st][k], base));
            most[0] = fmaxf(most[0], z[st][n][k].x);
            most[1] = fmaxf(most[1], z[st][n][k].y);
          }
#pragma unroll
        for (int r = 0; r < 2; ++r)
          high |= most[r] > kPBits + 1.5f || mx[n][r] - M(n, r) > 60.f;
      }
      return high;
    };
    if (__any_sync(0xffffffffu, exponents())) {
#pragma unroll
      for (int n = 0; n < kNt; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float top = row_max(mx[n][r]), to = fmaxf(M(n, r), top);
          float v = -INFINITY;  // the largest s + y, from `to`
#pragma unroll
          for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int k = 0; k < 2; ++k) v = fmaxf(v, (s[st][n][2 * k + r] - to) + lvs[st][k].x);
          move(n, r, top, to, row_max(v), 0.f);
        }
      exponents();
    }
#pragma unroll
    for (int n = 0; n < kNt; ++n) {
      const float2 minus_M = make_float2(-finite_or_0(M(n, 0)), -finite_or_0(M(n, 1)));
      float2 sum = make_float2(l[n][0], l[n][1]);
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 y = make_float2(s[st][n][2 * k], s[st][n][2 * k + 1]);
          const float2 t = __fadd2_rn(y, minus_M);
          sum = __fadd2_rn(sum, make_float2(ex2(t.x), ex2(t.y)));
          float2 w = make_float2(ex2(z[st][n][k].x), ex2(z[st][n][k].y));
          // Whatever the slot's scales are, and where no slot was attended yet.
          if (y.x == -INFINITY) w.x = 0.f;
          if (y.y == -INFINITY) w.y = 0.f;
          put_weights(st, n, k, w);
        }
      l[n][0] = sum.x;
      l[n][1] = sum.y;
    }
    follow();
  }

  template <bool kOwn, int kC>
  __device__ __forceinline__ void values(uint32_t stage) {
    constexpr int kW = D / 64;       // words of a V row a lane holds
    constexpr int kHalfT = kMt / 2;  // dims of a lane's share that are rows g: the first half
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const uint32_t from[2] = {stage + at_v[0], stage + at_v[1]}, from_s = stage + at_vs;
    each<2>([&](auto step) {
      constexpr int st = decltype(step)::value;
      uint32_t vw[4][kW];  // slots 2t, 2t+1, 2t+8, 2t+9
      each<4>([&](auto i) {
        constexpr int r = decltype(i)::value, row = 16 * st + 8 * (r >> 1);
        if constexpr (D == 128) {
          const uint2 w = lds64<row * (D / 2)>(from[r & 1]);
          vw[r][0] = w.x, vw[r][1] = w.y;
        } else {
          vw[r][0] = lds32<row * (D / 2)>(from[r & 1]);
        }
      });
      uint32_t sc[2];
      if constexpr (kOwn) {
        const uint16_t* vs = scales->v[D == 128 ? g >> 1 : g >> 2] + 16 * st + 2 * t4;
        sc[0] = *reinterpret_cast<const uint32_t*>(vs);
        sc[1] = *reinterpret_cast<const uint32_t*>(vs + 8);
      } else {
        const uint32_t c = (28u - rv) * 0x04000400u;
        each<2>([&](auto i) {
          constexpr int at = (16 * st + 8 * decltype(i)::value) * kGroups;
          sc[decltype(i)::value] = lds8<at>(from_s) * 0x0400u +
                                   (lds8<at + kGroups>(from_s) * 0x04000000u + c);
        });
      }
      // Halves of the slot pairs: [pair][dim of the lane's D / 8].
      uint32_t f[2][D / 8];
#pragma unroll
      for (int pr = 0; pr < 2; ++pr)
#pragma unroll
        for (int w = 0; w < kW; ++w) {
          const uint32_t x = vw[2 * pr][w], y = vw[2 * pr + 1][w];
          uint32_t even[4], odd[4];
          e2m1x8_to_half2(select_bits(0x0f0f0f0fu, x, y << 4), even);
          e2m1x8_to_half2(select_bits(0x0f0f0f0fu, x >> 4, y), odd);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            f[pr][8 * w + 2 * k] = hmul2(even[k], sc[pr]);
            f[pr][8 * w + 2 * k + 1] = hmul2(odd[k], sc[pr]);
          }
        }
      // Row g of m-tile i is dim (D/8) g + i, row g + 8 is dim (D/8) g + D/16 + i.
      static_assert(kHalfT * 2 == kMt && D / 16 == kMt, "");
#pragma unroll
      for (int i = 0; i < kMt; ++i) {
        const uint32_t fa[4] = {f[0][i], f[0][D / 16 + i], f[1][i], f[1][D / 16 + i]};
#pragma unroll
        for (int term = kTerms - 1; term >= 0; --term)
#pragma unroll
          for (int n = 0; n < kNt; ++n)
            mma16816(o[i][n], fa, pf[term][2 * kC + st][n][0], pf[term][2 * kC + st][n][1]);
      }
    });
  }

  // The warp's sums to shared memory.
  __device__ __forceinline__ void finish(float* osum, Stat* stat) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int n = 0; n < kNt; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float sum = l[n][r];  // the lane's slots'; the maxima are the warp's
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        const int row = warp * kTile + 8 * n + 2 * t4 + r;
        if (g == 0) stat[row] = Stat{M(n, r), D0(n, r), sum};
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int i = 0; i < kMt; i += 4)
            *reinterpret_cast<float4*>(osum + sum_at<D>(row, g * (D / 8) + half * (D / 16) + i)) =
                make_float4(o[i][n][2 * half + r], o[i + 1][n][2 * half + r],
                            o[i + 2][n][2 * half + r], o[i + 3][n][2 * half + r]);
      }
  }
};

// Number in the pool of a unit's chunk x (it fits: the entry points check), or
// kNoPage, which reads page 0 and attends nothing of it.
constexpr uint32_t kNoPage = 0xffffffffu;
__device__ __forceinline__ uint32_t chunk_at(const CacheAttnArgs& a, const Entry& e, int c, int x) {
  const int slot = e.win0 + x * kChunk;
  const int64_t page = cache_page(a.s, e.b, slot >> a.c.lb, a.c.n_pages, a.status);
  if (page < 0) return kNoPage;  // recorded
  return static_cast<uint32_t>((page * a.c.Hkv + c) << (a.c.lb - kChunkLog2)) +
         ((slot & (a.c.block - 1)) >> kChunkLog2);
}

template <int D, class Body>
__global__ void __launch_bounds__(kThreads, Body::kPerSm)
    cache4_attn_kernel(const Cache4AttnArgs a) {
  constexpr int kTile = Body::kTile, kStages = Body::kStages, kPair = Body::kPair;
  __shared__ uint32_t scan[kWarps];
  __shared__ uint32_t found[2];
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ Stat stat[kWarps * kTile];
  float* osum = reinterpret_cast<float*>(dyn);

  const Plan p = plan_of(a, kTile);
  let_next_start();
  const Scan sc = scan_entries<kWarps>(a, p, scan);
  const uint32_t W = sc.total * p.units;
  if (W == 0) return;
  const Cut cut = cut_of(a, p, W);
  if (blockIdx.x >= cut.P) return;
  const uint32_t begin = cta_begin(cut, blockIdx.x), end = cta_begin(cut, blockIdx.x + 1);
  // The entry that holds chunk `begin`, and its first chunk.
  each_entry<kWarps>(a, p, sc, scan, [&](int i, uint32_t before, uint32_t n) {
    if (begin >= before * p.units && begin < (before + n) * p.units) {
      found[0] = i;
      found[1] = before * p.units;
    }
  });
  __syncthreads();
  int i = static_cast<int>(found[0]);
  uint32_t base = found[1];  // first chunk of entry i
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t ring =
      static_cast<uint32_t>(__cvta_generic_to_shared(dyn)) + warp * Body::kRingBytes;
  constexpr uint32_t kRing = Body::kRingBytes, kStage = Body::kStageBytes;
  const typename Body::Place place = Body::place(a);

  Body body;
  for (uint32_t at = begin; at < end;) {
    Entry e = entry_at(a, i);
    while (at >= base + e.n_chunks * p.units) {
      base += e.n_chunks * p.units;
      e = entry_at(a, ++i);
    }
    const int u = (at - base) / static_cast<uint32_t>(e.n_chunks);
    const uint32_t u0 = base + u * e.n_chunks;
    const uint32_t stop = min(end, u0 + e.n_chunks);
    const int c = u / p.n_tiles, rt = u - c * p.n_tiles;
    // This CTA's chunks of the unit: [x0, x1) of its n_chunks; the warp's n pairs of
    // them, every kWarps-th from `mine` on, the last of all perhaps of one.
    const int x0 = static_cast<int>(at - u0), x1 = static_cast<int>(stop - u0);
    const int mine = x0 + warp * kPair;
    const int n = mine < x1 ? (x1 - mine + kWarps * kPair - 1) / (kWarps * kPair) : 0;
    // Pairs are looked up 32 ahead, a lane each, so that a copy never waits on the
    // table.
    uint32_t ahead[kPair];
    uint32_t dead[kPair][2];  // of the last 64 looked up, the chunks without a page
#pragma unroll
    for (int i = 0; i < kPair; ++i) dead[i][0] = dead[i][1] = 0;
    const auto start = [&](int k, uint32_t to) {
      if ((k & 31) == 0) {
#pragma unroll
        for (int i = 0; i < kPair; ++i) {
          const int x = mine + (k + lane) * kWarps * kPair + i;
          ahead[i] = x < x1 ? chunk_at(a, e, c, x) : 0;
          dead[i][0] = dead[i][1];
          dead[i][1] = __ballot_sync(0xffffffffu, ahead[i] == kNoPage);
          if (ahead[i] == kNoPage) ahead[i] = 0;
        }
      }
#pragma unroll
      for (int i = 0; i < kPair; ++i)
        if (i == 0 || mine + k * kWarps * kPair + i < x1)
          Body::copy(a, place, __shfl_sync(0xffffffffu, ahead[i], k & 31),
                     to + i * Body::kChunkBytes + lane * 16);
    };
#pragma unroll
    for (int k = 0; k < kStages; ++k) {
      if (k < n) start(k, ring + k * kStage);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    Body::load_rows(a, p, e, c, rt, dyn);
    __syncthreads();
    body.begin(dyn);
    const int pos0 = body.rows->pos[0];  // the first row's position, the last's
    const int pos1 = body.rows->pos[min(kTile, p.rows - rt * kTile) - 1];
    // Slots that every row attends, as first slots of pairs that lie in them; slots
    // that some row does.
    const int all0 = pos1 - a.window + 1, all1 = pos0 - (kPair * kChunk - 1);
    const int some0 = pos0 - a.window + 1, some1 = pos1;
    uint32_t stage = ring;
    int key0 = e.win0 + mine * kChunk;
    int x = mine;
    for (int k = 0; k < n; ++k, key0 += kWarps * kPair * kChunk, x += kWarps * kPair) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();
      uint32_t without = 0;
#pragma unroll
      for (int i = 0; i < kPair; ++i) without |= dead[i][0] | dead[i][1];
      const bool edge = without || key0 < all0 || key0 > all1 || x + kPair > x1;
      uint32_t live = (1u << kPair) - 1, off = 0;
      if (edge) {
        // Pair k was looked up with the latest 32, or with those before.
        const int newest = min(k + kStages, n) - 1;
        const bool now = (newest >> 5) == (k >> 5);
#pragma unroll
        for (int i = 0; i < kPair; ++i) {
          const uint32_t d = now ? dead[i][1] : dead[i][0];
          if ((d >> (k & 31) & 1) || x + i >= x1) live &= ~(1u << i);
          const int key = key0 + i * kChunk + lane;
          if (!(live >> i & 1) || key < some0 || key > some1) off |= 1u << i;
        }
        body.blank(stage, off);
      }
      if ((body.fits(stage) || body.refer(stage, off)) && body.level) {
        each<kPair>([&](auto i) {
          body.template scores<false, decltype(i)::value>(stage + decltype(i)::value *
                                                                      Body::kChunkBytes);
        });
        if (edge)
          body.template softmax_one<true>(a, key0, live);
        else
          body.template softmax_one<false>(a, key0, live);
        each<kPair>([&](auto i) {
          body.template values<false, decltype(i)::value>(stage + decltype(i)::value *
                                                                      Body::kChunkBytes);
        });
      } else {
#pragma unroll 1
        for (int i = 0; i < min(kPair, x1 - x); ++i) {
          const uint32_t from = stage + i * Body::kChunkBytes;
          body.read_scales(from);
          __syncwarp();
          body.template scores<true, 0>(from);
          body.softmax(a, key0 + i * kChunk, live >> i & 1);
          body.template values<true, 0>(from);
          __syncwarp();
        }
      }
      __syncwarp();
      if (k + kStages < n) start(k + kStages, stage);
      asm volatile("cp.async.commit_group;" ::: "memory");
      if constexpr (kStages == 2)
        stage = 2 * ring + kStage - stage;
      else
        stage = stage == ring + (kRing - kStage) ? ring : stage + kStage;
    }
    __syncthreads();
    body.finish(osum, stat);
    __syncthreads();
    const bool whole = x0 == 0 && x1 == e.n_chunks;
    join_warps<D, kTile>(a, p, e, c, rt, osum, stat, whole,
                         2 * static_cast<int64_t>(blockIdx.x) + (x0 == 0));
    __syncthreads();  // the sums make room for the next unit's chunks
    at = stop;
  }
}

template <int D, class Body>
cudaError_t launch_body4(const Cache4AttnArgs& a, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(cache4_attn_kernel<D, Body>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, Body::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_after(cache4_attn_kernel<D, Body>, dim3(a.n_ctas), kThreads, Body::kSmem, st, false,
                   a);
  if (e != cudaSuccess) return e;
  return launch_join<D, Body::kTile>(a, st);
}

template <int D>
cudaError_t launch_d(const Cache4AttnArgs& a, cudaStream_t st) {
  const int tile = a.tile;
  if (!a.in_bf16)
    return tile == 8 ? launch_body4<D, Body4<D, 1, 2>>(a, st)
                     : launch_body4<D, Body4<D, 2, 2>>(a, st);
  return tile == 8    ? (a.pairs ? launch_body4<D, Body4<D, 1, 1, 2>>(a, st)
                                 : launch_body4<D, Body4<D, 1, 1>>(a, st))
         : tile == 16 ? launch_body4<D, Body4<D, 2, 1>>(a, st)
                      : launch_body4<D, Body4<D, 4, 1>>(a, st);
}

}  // namespace

// Tiles of 8, 16 or (bf16) 32 rows: as many as the rows fill, but two of 16 for 32
// over few slots: a CTA's start and end with 32 rows cost more than the second read
// of the slots (four tokens of 64 heads on 8 of each of 16 sequences: over 32 slots
// 24.8 us with 32 rows and 18.1 with 16, over 4096 53.7 and 52.0, over 16384 139 and
// 150).
int cache4_attn_tile_rows(int rows, int64_t slots, int in_bf16) {
  return rows <= 8 ? 8 : rows <= 16 || !in_bf16 || slots <= 6144 ? 16 : 32;
}
// Pairs of chunks from 96 chunks a CTA on, as many at most: a pair takes 5 to 8 % less
// time than two chunks, but a range of few chunks is no whole number of pairs for
// every warp, and the longer code is read for the first time (one token of 64 heads on
// 8; 16 sequences: over 1024 slots 17.4 us with pairs and 16.2 without, over 4096 27.0
// and 25.2, over 8192 40.2 and 40.0, over 16384 61.5 and 62.9; 64 sequences of 16K to
// 32K slots 286 and 305).
bool cache4_attn_pairs(int64_t chunks, int max_ctas) { return chunks >= int64_t(96) * max_ctas; }
int cache4_attn_max_ctas(int tile_rows, int in_bf16) {
  return kSms * (tile_rows == 8    ? Body4<128, 1, 1>::kPerSm
                 : tile_rows == 32 ? Body4<128, 4, 1>::kPerSm
                 : in_bf16         ? Body4<128, 2, 1>::kPerSm
                                   : Body4<128, 2, 2>::kPerSm);
}

cudaError_t launch_cache4_attn(const Cache4AttnArgs& a, cudaStream_t st) {
  return a.c.d == 128 ? launch_d<128>(a, st) : launch_d<64>(a, st);
}

}  // namespace msa
