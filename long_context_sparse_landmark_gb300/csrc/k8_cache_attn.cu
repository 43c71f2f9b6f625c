// K8: attention of a few query tokens over the 8-bit KV cache, in full,
// over a window, or over a window and selected blocks.
//
// Mathematics, per query row (position p, head h of KV group c), over its
// slots j, in log2 units: s_j = scale log2e <q, code_j> kscale(j), v_j = log2
// vscale(j); out = sum_j 2^{s_j + v_j} code_j / sum_j 2^{s_j}.  The value scale
// goes into the exponent of the weights that meet the raw codes: w_j = 2^{(s_j -
// M) + (v_j - D)}, with M the largest s so far (to 60), the denominator's
// reference, and M + D the largest s + v (to 1.5), the output's.  Kept as an
// offset D of M, so that a large score does not round the value scale away; M
// never falls, so that neither sum leaves fp32 where the largest s and the
// largest s + v are slots far apart.  All sums are fp32.
//
// The work is read once: 2 d bytes a slot and KV head, shared by the group's
// rows, so HBM bounds it: 64 sequences of 16K to 32K tokens, 64 heads on 8 of
// 128, take 495 us, 6.66 TB/s (98 % of a measured copy's 6.79).  The slots of
// all (sequence, KV head, row tile) units form one list of 32-slot chunks that
// is cut into equal ranges, one a CTA, whatever the lengths are (they are only
// known on the device); where a cut falls inside a unit the parts are joined
// by a second kernel, which starts while this one drains.
//
// bf16 rows run on the tensor cores (mma.sync, fp16 operands): codes turn
// into halves exactly, a row of q is scaled by a power of two so that it
// does too (an element 2^-31 of the row's largest and smaller is rounded),
// and the weights are halves with 11 bits, scaled to use the whole range
// (2^14 for the largest, so 2^-28 of it still has full precision).  Keys
// are the MMA's 16 rows and query rows its 8 columns, so a group of 8 heads
// wastes nothing; a warp's chunks come by cp.async into a ring of its own,
// and a lane's 16-byte piece of a row is its share of four k-steps, the d (or
// slot) index permuted alike on both operands.  tcgen05 would need the codes
// widened in shared memory first and 64 or 128 rows to fill its M; one token
// needs 32 operations a byte, far below what either unit does.
//   Up to 8, 16 or 32 rows share a read.  At 32 (four tokens of eight heads)
// the latencies of the loop's some 950 instructions a chunk on 8 warps an SM
// bound it (tensor pipe 21 % busy, issue slots 23 %): 16 sequences of 17K to 32K
// slots take 139 us with one token (6.05 TB/s), 143 with two, 208 with four (362
// as two passes of 16 rows, when four took 218).  Short calls are bound by
// latency: 32K tokens of one KV head take 11.0 us with the join, 6.4 of them here;
// a part's first pass through the code, cold in the instruction cache, costs
// more than its chunks.
// fp32 rows run on the CUDA cores with fp32 arithmetic throughout: packed
// multiply-adds, 8 rows a read.  8 sequences of 20K to 32K slots, 64 heads on 8 of
// 128, take 247 us, 26 TFLOP/s of the 80 that the fp32 lanes have.  No unit is
// full (issue slots 37 %, the shared-memory pipe 53 %, fp32 lanes 35 %): the
// registers allow 12 warps an SM, which wait for loads (1.7 warps a scheduler and
// issue), fixed latencies (1.3) and shared memory (1.1).
#include <math.h>
#include "cache_attn.cuh"

namespace msa {
namespace {

// What a warp knows of the chunk it works on.
struct Chunk {
  int64_t at;    // first slot's row in the codes [n_pages * Hkv * block, d]
  int key0;      // first slot
  float ks, lvs;  // scale of K, log2 of that of V
  bool on;       // false: nothing to attend (a selection shorter than top_k)
  bool window;   // of the window part: rows' own limits apply
};

// Chunks x, x + kWarps, ... of a unit, read 32 ahead: lane l holds the page
// and scales of chunk x + l * kWarps, so that a chunk's loads never wait on
// the table.
struct Ahead {
  int64_t at;
  int key0;
  float ks, lvs;
  int flags;
};

__device__ __forceinline__ Ahead look_ahead(const CacheAttnArgs& a, const Entry& e, int c,
                                            int x, int end) {
  Ahead r;
  r.at = 0;
  r.key0 = 0;
  r.ks = r.lvs = 0.f;
  r.flags = 0;
  if (x >= end) return r;
  const int per_log2 = a.c.lb - kChunkLog2, x_win = e.n_sel << per_log2;
  int slot;
  if (x < x_win) {
    const int64_t u = (static_cast<int64_t>(e.b) * a.T + e.t) * a.c.Hkv + c;
    const int i = x >> per_log2;
    const int32_t cnt = a.cnt[u], chosen = a.sel[u * a.top_k + i];
    if (i >= sel_count_checked(cnt, a.top_k, e.n_cand, a.status)) return r;
    const int blk = sel_block_checked(chosen, e.n_cand, a.status);
    slot = (blk << a.c.lb) + (x - (i << per_log2)) * kChunk;
    r.flags = 1;
  } else {
    slot = e.win0 + (x - x_win) * kChunk;
    r.flags = 3;
  }
  const int j = slot >> a.c.lb;
  int64_t page = cache_page(a.s, e.b, j, a.c.n_pages, a.status);
  if (page < 0) {  // recorded; read a page that exists
    page = 0;
    r.flags = 0;
  }
  r.key0 = slot;
  const int64_t head = page * a.c.Hkv + c;
  r.at = (head << a.c.lb) + (slot & (a.c.block - 1));
  r.ks = a.c.k_scale[head];
  const float vs = a.c.v_scale[head];
  r.lvs = vs == 0.f ? kLogZero : log2f(vs);
  return r;
}

__device__ __forceinline__ Chunk chunk_of(const Ahead& r, int src) {
  Chunk c;
  c.key0 = __shfl_sync(0xffffffffu, r.key0, src);
  c.at = __shfl_sync(0xffffffffu, r.at, src);
  c.ks = __shfl_sync(0xffffffffu, r.ks, src);
  c.lvs = __shfl_sync(0xffffffffu, r.lvs, src);
  const int f = __shfl_sync(0xffffffffu, r.flags, src);
  c.on = f & 1;
  c.window = f & 2;
  return c;
}

// ---- the bodies ------------------------------------------------------------

// Tensor cores: 8 * kNt query rows.
template <int D, int kNt>
struct MmaBody {
  static constexpr int kTile = 8 * kNt;
  // 12 warps an SM with 16 KB of chunks under way each, or 8 with 24 KB; the
  // rows of four tiles no longer fit the registers.
  static constexpr int kPerSm = kNt == 1 ? 3 : 2;
  static constexpr int kStages = (kNt == 1 ? 2 : 3) * (D == 128 ? 1 : 2);
  static constexpr bool kQShared = kNt > 2;
  static constexpr int kStageBytes = 2 * kChunk * D;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kKs = D / 16;   // k-steps over d
  static constexpr int kMt = D / 16;   // 16-row tiles of O^T
  static constexpr int kKw = D / 16;   // words of a K row a lane holds
  static constexpr int kVw = D / 32;   // words of a V row a lane holds

  uint32_t q[kQShared ? 1 : kKs][kQShared ? 1 : kNt][2];
  float qs[kNt][2];   // score scale of rows 2t, 2t+1 (log2 units)
  float o[kMt][kNt][4];
  float l[kNt][2], M[kNt][2], D0[kNt][2];  // l in units of 2^M, o of 2^{M + D0 - kPBits}

  // Rows of a unit, in shared memory for all its warps: their fragments
  // [k-step][tile][lane], score scales and positions.
  struct Rows {
    uint2 q[kKs * kNt * 32];
    float scale[kTile];
    int pos[kTile];
  };
  static constexpr int kSmem = kWarps * kRingBytes + static_cast<int>(sizeof(Rows));
  static_assert(kWarps * kRingBytes >= kWarps * kTile * (D + 4) * 4, "sums must fit the rings");

  // The CTA writes them: a thread takes 16-byte pieces of rows.
  __device__ __forceinline__ static void load_rows(const CacheAttnArgs& a, const Plan& p,
                                                   const Entry& e, int c, int rt, uint8_t* smem) {
    constexpr int kP = D / 8;
    Rows& rows = *reinterpret_cast<Rows*>(smem + kWarps * kRingBytes);
#pragma unroll 1
    for (int i = threadIdx.x; i < kTile * kP; i += kThreads) {  // whole warps
      const int r = i / kP, pc = i - r * kP, m = rt * kTile + r;
      int t, h;
      row_of(a, e, c, min(m, p.rows - 1), &t, &h);
      uint4 x = make_uint4(0, 0, 0, 0);
      if (m < p.rows)
        x = *reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(a.q) +
            ((static_cast<int64_t>(e.b) * a.T + t) * a.Hq + h) * D + 8 * pc);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      float v[8], mx = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(w[k] << 16);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        mx = fmaxf(mx, fmaxf(fabsf(v[2 * k]), fabsf(v[2 * k + 1])));
      }
#pragma unroll
      for (int o2 = 1; o2 < kP; o2 <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o2));
      // 2^k brings the row's largest magnitude to [2^14, 2^15).
      int k = mx > 0.f ? 14 + 127 - static_cast<int>(__float_as_uint(mx) >> 23) : 0;
      k = k > 100 ? 100 : k;
      const float up = pow2i(k);
      // d = 64 hf + 16 t4 + 4 w + 0..3 is word w of lane t4's piece: k-step 4 hf + w.
      const int ks = 4 * (pc >> 3) + 2 * (pc & 1);
      uint2* to = rows.q + (ks * kNt + (r >> 3)) * 32 + (r & 7) * 4 + ((pc & 7) >> 1);
      to[0] = make_uint2(half2_of(v[0] * up, v[1] * up), half2_of(v[2] * up, v[3] * up));
      to[kNt * 32] = make_uint2(half2_of(v[4] * up, v[5] * up), half2_of(v[6] * up, v[7] * up));
      if (pc == 0) {
        rows.scale[r] = a.scale * kLog2e * pow2i(-k);
        rows.pos[r] = e.len - a.T + t;
      }
    }
  }

  const Rows* rows;

  __device__ __forceinline__ void begin(const uint8_t* smem) {
    const int lane = threadIdx.x & 31, t4 = lane & 3;
    rows = reinterpret_cast<const Rows*>(smem + kWarps * kRingBytes);
#pragma unroll
    for (int n = 0; n < kNt; ++n) {
      if constexpr (!kQShared) {
#pragma unroll
        for (int ks = 0; ks < kKs; ++ks) {
          const uint2 x = rows->q[(ks * kNt + n) * 32 + lane];
          q[ks][n][0] = x.x;
          q[ks][n][1] = x.y;
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        qs[n][r] = rows->scale[8 * n + 2 * t4 + r];
        M[n][r] = -INFINITY;
        l[n][r] = D0[n][r] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kMt; ++i)
#pragma unroll
      for (int n = 0; n < kNt; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][n][k] = 0.f;
  }

  // A warp's chunks pass through a ring of its own in shared memory: K and V
  // codes as [32][D] each, 16-byte pieces (and for d = 64 rows of V) moved
  // about so that the fragment reads below meet no bank twice.
  __device__ __forceinline__ static int k_at(int row, int piece) {
    return D == 128 ? row * 128 + ((piece ^ ((row & 1) << 2)) << 4) : row * 64 + (piece << 4);
  }
  __device__ __forceinline__ static int v_at(int row, int piece) {
    return kChunk * D + (D == 128 ? row * 128 + ((piece ^ (row & 6)) << 4)
                                  : (row ^ ((row >> 2) & 1)) * 64 + ((piece ^ (row & 2)) << 4));
  }
  // Starts the copy of the chunk whose first slot is row `at` of the codes.
  __device__ __forceinline__ static void copy(const CacheAttnArgs& a, int64_t at, uint8_t* stage) {
    constexpr int kPer = D / 16;        // pieces a row
    constexpr int kStep = 32 / kPer;    // rows the warp copies at a time
    const int lane = threadIdx.x & 31, piece = lane % kPer, row0 = lane / kPer;
    if (!MSA_IN_RANGE(at, kChunk, a.c.n_pages * a.c.Hkv * a.c.block, a.status)) return;
    const uint8_t* k = a.c.k_codes + at * D + lane * 16;
    const uint8_t* v = a.c.v_codes + at * D + lane * 16;
#pragma unroll
    for (int i = 0; i < kChunk / kStep; ++i)
      copy_async16(stage + k_at(row0 + i * kStep, piece), k + i * 512);
#pragma unroll
    for (int i = 0; i < kChunk / kStep; ++i)
      copy_async16(stage + v_at(row0 + i * kStep, piece), v + i * 512);
  }

  uint32_t kw[2][2][kKw];   // [16-slot step][slot g / g + 8][word]
  uint32_t vw[2][4][kVw];   // [16-slot step][slot 2t, 2t+1, 2t+8, 2t+9][word]

  __device__ __forceinline__ void read_k(const uint8_t* stage) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf) {
          const uint4 w =
              *reinterpret_cast<const uint4*>(stage + k_at(16 * s + 8 * r + g, 4 * hf + t4));
          kw[s][r][4 * hf] = w.x;
          kw[s][r][4 * hf + 1] = w.y;
          kw[s][r][4 * hf + 2] = w.z;
          kw[s][r][4 * hf + 3] = w.w;
        }
  }
  __device__ __forceinline__ void read_v(const uint8_t* stage) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * s + 8 * (r >> 1) + 2 * t4 + (r & 1);
        if constexpr (D == 128) {
          const uint4 w = *reinterpret_cast<const uint4*>(stage + v_at(row, g));
          vw[s][r][0] = w.x;
          vw[s][r][1] = w.y;
          vw[s][r][2] = w.z;
          vw[s][r][3] = w.w;
        } else {
          const uint2 w =
              *reinterpret_cast<const uint2*>(stage + v_at(row, g >> 1) + 8 * (g & 1));
          vw[s][r][0] = w.x;
          vw[s][r][1] = w.y;
        }
      }
  }

  float s[2][kNt][4];

  __device__ __forceinline__ void scores() {
#pragma unroll
    for (int st = 0; st < 2; ++st)
#pragma unroll
      for (int n = 0; n < kNt; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[st][n][k] = 0.f;
#pragma unroll
    for (int ks = 0; ks < kKs; ++ks) {
      uint32_t b[kNt][2];
#pragma unroll
      for (int n = 0; n < kNt; ++n) {
        if constexpr (kQShared) {
          const uint2 x = rows->q[(ks * kNt + n) * 32 + (threadIdx.x & 31)];
          b[n][0] = x.x;
          b[n][1] = x.y;
        } else {
          b[n][0] = q[ks][n][0];
          b[n][1] = q[ks][n][1];
        }
      }
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const uint32_t fa[4] = {e4m3x2_to_half2(static_cast<uint16_t>(kw[st][0][ks])),
                                e4m3x2_to_half2(static_cast<uint16_t>(kw[st][1][ks])),
                                e4m3x2_to_half2(static_cast<uint16_t>(kw[st][0][ks] >> 16)),
                                e4m3x2_to_half2(static_cast<uint16_t>(kw[st][1][ks] >> 16))};
#pragma unroll
        for (int n = 0; n < kNt; ++n) mma16816(s[st][n], fa, b[n][0], b[n][1]);
      }
    }
  }

  // Softmax of the chunk's scores into halves pf[step][nt][b0, b1], and the
  // running sums.  kEdge: some slot is masked for some row.
  uint32_t pf[2][kNt][2];

  template <bool kEdge, bool kWeights>
  __device__ __forceinline__ void softmax(const CacheAttnArgs& a, const Plan& p, const Entry& e,
                                          int c, int rt, const Chunk& x) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    // The references are not kept up to the last bit: a weight may exceed 2^14
    // by a factor 2^1.5 (the half's range allows it) and a term of the
    // denominator 1 by 2^60, so that most chunks move neither them nor the sums,
    // and the lanes need not agree on a maximum.
    float mx[kNt][2];
    bool rise = false;
#pragma unroll
    for (int n = 0; n < kNt; ++n) {
      // Rows 2t and 2t + 1 side by side, as the fragments have them.
      const float2 f = make_float2(qs[n][0] * x.ks, qs[n][1] * x.ks);  // >= 0, or NaN
      int pos[2] = {0, 0};
      if (kEdge) {
        pos[0] = rows->pos[8 * n + 2 * t4];
        pos[1] = rows->pos[8 * n + 2 * t4 + 1];
      }
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 y =
              __fmul2_rn(make_float2(s[st][n][2 * k], s[st][n][2 * k + 1]), f);
          s[st][n][2 * k] = y.x;
          s[st][n][2 * k + 1] = y.y;
          if (kEdge) {
            const int key = x.key0 + 16 * st + 8 * k + g;
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (!x.on || (x.window && (key > pos[r] || pos[r] - key >= a.window)))
                s[st][n][2 * k + r] = -INFINITY;
          }
        }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[n][r] = fmaxf(fmaxf(s[0][n][r], s[0][n][2 + r]), fmaxf(s[1][n][r], s[1][n][2 + r]));
        const float up = mx[n][r] - M[n][r];
        rise |= up + (x.lvs - D0[n][r]) > 1.5f || up > 60.f;
      }
      if constexpr (kWeights) {
        // For the weights pass: [slot][row], rows padded to even.
        const int even = (p.rows + 1) & ~1;
        const int row = rt * kTile + 8 * n + 2 * t4;
        if (row < even) {
          const int64_t slots = static_cast<int64_t>(a.s.max_blocks) * a.c.block;
          float* to = a.scores + ((static_cast<int64_t>(e.b) * a.c.Hkv + c) * slots + x.key0) * even;
          if (MSA_IN_RANGE(x.key0, kChunk, slots, a.status))
#pragma unroll
            for (int st = 0; st < 2; ++st)
#pragma unroll
              for (int k = 0; k < 2; ++k)
                *reinterpret_cast<float2*>(to + static_cast<int64_t>(16 * st + 8 * k + g) * even +
                                           row) =
                    make_float2(s[st][n][2 * k], s[st][n][2 * k + 1]);
        }
      }
    }
    if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
      for (int n = 0; n < kNt; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float top = mx[n][r];
#pragma unroll
          for (int o2 = 4; o2 < 32; o2 <<= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o2));
          const float up = top - M[n][r];
          if (up + (x.lvs - D0[n][r]) > 0.f || up > 60.f) {
            const float to = fmaxf(M[n][r], top), kept = D0[n][r] - (to - M[n][r]);
            const float off = fmaxf(kept, x.lvs + (top - to));  // kept: the output's unit stays
            const float down = ex2(kept - off);
            l[n][r] *= ex2(M[n][r] - to);
#pragma unroll
            for (int i = 0; i < kMt; ++i) {
              o[i][n][r] *= down;
              o[i][n][2 + r] *= down;
            }
            M[n][r] = to;
            D0[n][r] = off;
          }
        }
    }
#pragma unroll
    for (int n = 0; n < kNt; ++n) {
      float pv[2][4];
      const float2 minus_M = make_float2(-finite_or_0(M[n][0]), -finite_or_0(M[n][1]));
      const float2 v = make_float2(x.lvs - D0[n][0], x.lvs - D0[n][1]);
      const float2 base = make_float2(kPBits + v.x, kPBits + v.y);
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 y = make_float2(s[st][n][2 * k], s[st][n][2 * k + 1]);
          const float2 z = __fadd2_rn(__fadd2_rn(y, minus_M), base);
          float2 w = make_float2(ex2(z.x), ex2(z.y));
          if (kEdge) {  // whatever the block's scales are
            if (y.x == -INFINITY) w.x = 0.f;
            if (y.y == -INFINITY) w.y = 0.f;
          }
          pv[st][2 * k] = w.x;
          pv[st][2 * k + 1] = w.y;
          sum = __fadd2_rn(sum, w);
        }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float mM = r ? minus_M.y : minus_M.x, sr = r ? sum.y : sum.x;
        // The denominator: the weights with the value scale taken out again, ...
        float part = sr * ex2(-(r ? base.y : base.x));
        if (kEdge && sr == 0.f) part = 0.f;
        // ... unless they are too small to tell it: values 2^60 below other
        // blocks', or not numbers.
        if (!((mx[n][r] + mM) + (r ? v.y : v.x) >= -60.f)) {
          part = 0.f;
#pragma unroll
          for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int k = 0; k < 2; ++k) part += ex2(s[st][n][2 * k + r] + mM);
        }
        l[n][r] += part;
      }
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        pf[st][n][0] = transpose8x8(half2_of(pv[st][0], pv[st][1]));
        pf[st][n][1] = transpose8x8(half2_of(pv[st][2], pv[st][3]));
      }
    }
  }

  // A slot no row may attend holds anything, NaN codes too: its weight is 0,
  // its value must be as well.
  __device__ __forceinline__ void clear_masked(const Chunk& x, int first, int last) {
    const int t4 = threadIdx.x & 3;
#pragma unroll
    for (int st = 0; st < 2; ++st)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int key = x.key0 + 16 * st + 8 * (r >> 1) + 2 * t4 + (r & 1);
        if (!x.on || (x.window && (key < first || key > last))) {
#pragma unroll
          for (int w = 0; w < kVw; ++w) vw[st][r][w] = 0u;
        }
      }
  }

  __device__ __forceinline__ void values() {
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      // Row index g of m-tile i is dim (D/8) g + i, index g + 8 is dim
      // (D/8) g + D/16 + i: byte i and byte i + D/16 of the lane's piece.
#pragma unroll
      for (int w = 0; w < kVw / 2; ++w) {
        const int w2 = w + kVw / 2;
        uint32_t f01[2][2], f23[2][2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t sel = half ? 0x7362u : 0x5140u;
          f01[0][half] = __byte_perm(vw[st][0][w], vw[st][1][w], sel);
          f01[1][half] = __byte_perm(vw[st][0][w2], vw[st][1][w2], sel);
          f23[0][half] = __byte_perm(vw[st][2][w], vw[st][3][w], sel);
          f23[1][half] = __byte_perm(vw[st][2][w2], vw[st][3][w2], sel);
        }
#pragma unroll
        for (int byte = 0; byte < 4; ++byte) {
          const int half = byte >> 1, sh = (byte & 1) * 16;
          const uint32_t fa[4] = {e4m3x2_to_half2(static_cast<uint16_t>(f01[0][half] >> sh)),
                                  e4m3x2_to_half2(static_cast<uint16_t>(f01[1][half] >> sh)),
                                  e4m3x2_to_half2(static_cast<uint16_t>(f23[0][half] >> sh)),
                                  e4m3x2_to_half2(static_cast<uint16_t>(f23[1][half] >> sh))};
#pragma unroll
          for (int n = 0; n < kNt; ++n)
            mma16816(o[4 * w + byte][n], fa, pf[st][n][0], pf[st][n][1]);
        }
      }
    }
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
        if (g == 0) stat[row] = Stat{M[n][r], D0[n][r], sum};
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

// CUDA cores, fp32 throughout: 8 query rows, a lane a slot for the scores
// and D/32 dims for the output.
template <int D>
struct SimtBody {
  static constexpr int kTile = 8;
  static constexpr int kPerSm = 3;
  static constexpr int kDl = D / 32;
  // The warps' sums, then q rows [8][D] for the CTA and weights [32][8] for
  // each warp.
  static constexpr int kSums = kWarps * kTile * (D + 4) * 4;
  static constexpr int kSmem = kSums + (kTile * D + kTile + kWarps * kChunk * kTile) * 4;

  float2 o[kTile / 2][kDl];  // rows 2i, 2i + 1
  float l[kTile], M[kTile], D0[kTile];  // l: the lane's slots, in units of 2^M; o: of 2^{M + D0}
  float* qsm;
  float* psm;

  // The CTA writes the unit's rows and their positions.
  __device__ __forceinline__ static void load_rows(const CacheAttnArgs& a, const Plan& p,
                                                   const Entry& e, int c, int rt, uint8_t* smem) {
    float* q = reinterpret_cast<float*>(smem + kSums);
    int* pos = reinterpret_cast<int*>(q + kTile * D);
#pragma unroll 1
    for (int i = threadIdx.x; i < kTile * D / 4; i += kThreads) {
      const int r = i / (D / 4), dim = (i - r * (D / 4)) * 4, row = rt * kTile + r;
      int t, h;
      row_of(a, e, c, min(row, p.rows - 1), &t, &h);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < p.rows)
        v = *reinterpret_cast<const float4*>(
            static_cast<const float*>(a.q) +
            ((static_cast<int64_t>(e.b) * a.T + t) * a.Hq + h) * D + dim);
      *reinterpret_cast<float4*>(q + r * D + dim) = v;
      if (dim == 0) pos[r] = e.len - a.T + t;
    }
  }

  const int* pos;

  __device__ __forceinline__ void begin(uint8_t* smem) {
    qsm = reinterpret_cast<float*>(smem + kSums);
    pos = reinterpret_cast<const int*>(qsm + kTile * D);
    psm = qsm + kTile * D + kTile + (threadIdx.x >> 5) * kChunk * kTile;
#pragma unroll
    for (int r = 0; r < kTile; ++r) {
      M[r] = -INFINITY;
      l[r] = D0[r] = 0.f;
    }
#pragma unroll
    for (int r = 0; r < kTile / 2; ++r)
#pragma unroll
      for (int k = 0; k < kDl; ++k) o[r][k] = make_float2(0.f, 0.f);
  }

  // 8 slots' codes of the lane's dims.
  __device__ __forceinline__ static void load_v(const uint8_t* at, uint32_t* w) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (D == 128)
        w[j] = __ldg(reinterpret_cast<const uint32_t*>(at + j * D));
      else
        w[j] = __ldg(reinterpret_cast<const uint16_t*>(at + j * D));
    }
  }

  __device__ __forceinline__ void chunk(const CacheAttnArgs& a, const Plan& p, const Entry& e,
                                        int c, int rt, const Chunk& x) {
    const int lane = threadIdx.x & 31;
    if (!MSA_IN_RANGE(x.at, kChunk, a.c.n_pages * a.c.Hkv * a.c.block, a.status)) return;
    const uint4* krow = reinterpret_cast<const uint4*>(a.c.k_codes + (x.at + lane) * D);
    const uint8_t* vbase = a.c.v_codes + x.at * D + lane * kDl;
    // Even and odd dims side by side; a piece of the row is under way while
    // the one before is multiplied, and eight slots' values likewise.
    float2 s2[kTile];
#pragma unroll
    for (int r = 0; r < kTile; ++r) s2[r] = make_float2(0.f, 0.f);
    uint4 w0 = __ldg(krow), w1 = __ldg(krow + 1);
#pragma unroll 1
    for (int d0 = 0; d0 < D; d0 += 16) {
      const uint32_t w[4] = {w0.x, w0.y, w0.z, w0.w};
      w0 = w1;
      if (d0 + 32 < D) w1 = __ldg(krow + d0 / 16 + 2);
      float kf[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) e4m3x4_to_float(w[i], kf + 4 * i);
#pragma unroll
      for (int r = 0; r < kTile; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 qv = *reinterpret_cast<const float4*>(qsm + r * D + d0 + 4 * i);
          s2[r] = __ffma2_rn(make_float2(qv.x, qv.y), make_float2(kf[4 * i], kf[4 * i + 1]), s2[r]);
          s2[r] =
              __ffma2_rn(make_float2(qv.z, qv.w), make_float2(kf[4 * i + 2], kf[4 * i + 3]), s2[r]);
        }
    }
    uint32_t vw[8];
    load_v(vbase, vw);
    float s[kTile];
#pragma unroll
    for (int r = 0; r < kTile; ++r) s[r] = s2[r].x + s2[r].y;
    const int key = x.key0 + lane;
    // Scores in log2 units as a float and what it leaves, and references
    // rounded up to whole numbers: the exponentials see differences whose error
    // goes by their own size, and a change of reference scales by a power of two.
    const float c_hi = a.scale * kLog2e;
    const float c_lo = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634 - c_hi);
    float lo[kTile];
    bool any = false;
#pragma unroll
    for (int r = 0; r < kTile; ++r) {
      const bool in = x.on && (!x.window || (key <= pos[r] && pos[r] - key < a.window));
      any |= in;
      const float y = s[r] * x.ks, t = y * c_hi;
      // Beyond 2^20 what is left is no fraction any more.
      lo[r] = in && fabsf(t) < 1048576.f ? fmaf(y, c_hi, -t) + y * c_lo : 0.f;
      s[r] = in ? t : -INFINITY;
    }
    if (a.weights) {
      const int even = (p.rows + 1) & ~1;
      const int64_t slots = static_cast<int64_t>(a.s.max_blocks) * a.c.block;
      float* to = a.scores +
                  ((static_cast<int64_t>(e.b) * a.c.Hkv + c) * slots + key) * even + rt * kTile;
#pragma unroll
      for (int r = 0; r < kTile; ++r)
        if (rt * kTile + r < even && MSA_IN_RANGE(key, 1, slots, a.status)) to[r] = s[r] + lo[r];
    }
    // References as in the other body, but whole numbers, so that a move of
    // either is exact; a weight may exceed 1 by 2^20 before they do.
    bool rise = false, apart = false;
#pragma unroll
    for (int r = 0; r < kTile; ++r) {
      const float up = s[r] - M[r], v = x.lvs - D0[r];
      rise |= up + v > 20.f || up > 60.f;
    }
    if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
      for (int r = 0; r < kTile; ++r) {
        float top = s[r];
#pragma unroll
        for (int x2 = 16; x2 > 0; x2 >>= 1)
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x2));
        top = ceilf(top);
        const float up = top - M[r];
        if (up + (x.lvs - D0[r]) > 0.f || up > 60.f) {
          const float to = fmaxf(M[r], top), kept = D0[r] - (to - M[r]);
          const float off = ceilf(fmaxf(kept, x.lvs + (top - to)));
          const float down = exp2f(kept - off);
          l[r] *= exp2f(M[r] - to);
#pragma unroll
          for (int k = 0; k < kDl; ++k) (r & 1 ? o[r / 2][k].y : o[r / 2][k].x) *= down;
          M[r] = to;
          D0[r] = off;
        }
      }
    }
    float pw[kTile];
#pragma unroll
    for (int r = 0; r < kTile; ++r) apart |= fabsf(x.lvs - D0[r]) > 60.f;
#pragma unroll
    for (int r = 0; r < kTile; ++r) {
      const float y = (s[r] - finite_or_0(M[r])) + lo[r], e = exp2f(y);
      l[r] += e;
      // Value scales 2^60 apart: the two exponents go together.
      const float w = apart ? exp2f(y + (x.lvs - D0[r])) : e * exp2f(x.lvs - D0[r]);
      pw[r] = s[r] == -INFINITY ? 0.f : w;
    }
    __syncwarp();
    *reinterpret_cast<float4*>(psm + lane * kTile) = make_float4(pw[0], pw[1], pw[2], pw[3]);
    *reinterpret_cast<float4*>(psm + lane * kTile + 4) = make_float4(pw[4], pw[5], pw[6], pw[7]);
    const uint32_t held = __ballot_sync(0xffffffffu, any);
    __syncwarp();
#pragma unroll 1
    for (int j0 = 0; j0 < kChunk; j0 += 8) {
      uint32_t cur[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) cur[j] = held >> (j0 + j) & 1 ? vw[j] : 0u;  // masked: anything
      if (j0 + 8 < kChunk) load_v(vbase + (j0 + 8) * D, vw);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float vf[4];
        if constexpr (D == 128) {
          e4m3x4_to_float(cur[j], vf);
        } else {
          const float2 f = e4m3x2_to_float2(static_cast<uint16_t>(cur[j]));
          vf[0] = f.x;
          vf[1] = f.y;
        }
        const float4 p0 = *reinterpret_cast<const float4*>(psm + (j0 + j) * kTile);
        const float4 p1 = *reinterpret_cast<const float4*>(psm + (j0 + j) * kTile + 4);
        const float2 pr[kTile / 2] = {make_float2(p0.x, p0.y), make_float2(p0.z, p0.w),
                                      make_float2(p1.x, p1.y), make_float2(p1.z, p1.w)};
#pragma unroll
        for (int k = 0; k < kDl; ++k)
#pragma unroll
          for (int r = 0; r < kTile / 2; ++r)
            o[r][k] = __ffma2_rn(pr[r], make_float2(vf[k], vf[k]), o[r][k]);
      }
    }
  }

  __device__ __forceinline__ void finish(float* osum, Stat* stat) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int r = 0; r < kTile; ++r) {
      float sum = l[r];
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      // (a weight of 1 is 2^0 here, 2^kPBits in the other body)
      if (lane == 0) stat[warp * kTile + r] = Stat{M[r], D0[r] + kPBits, sum};
#pragma unroll
      for (int k = 0; k < kDl; ++k) 
        osum[sum_at<D>(warp * kTile + r, lane * kDl + k)] = r & 1 ? o[r / 2][k].y : o[r / 2][k].x;
    }
  }
};

template <class Body>
struct IsMma {
  static constexpr bool value = false;
};
template <int D, int kNt>
struct IsMma<MmaBody<D, kNt>> {
  static constexpr bool value = true;
};

template <int D, class Body>
__global__ void __launch_bounds__(kThreads, Body::kPerSm) cache_attn_kernel(const CacheAttnArgs a) {
  constexpr int kTile = Body::kTile;
  __shared__ uint32_t scan[kWarps];
  __shared__ uint32_t found[2];
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ Stat stat[kWarps * kTile];
  __shared__ __align__(16) float4 info[kWarps][8];  // of a stage: K scale, log2 of V's, first slot, flags
  float* osum = reinterpret_cast<float*>(dyn);

  const Plan p = plan_of(a, kTile);
  let_next_start();
  wait_for_inputs();
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
    // This CTA's chunks of the unit: [x0, x1) of its n_chunks.
    const int x0 = static_cast<int>(at - u0), x1 = static_cast<int>(stop - u0);

    if constexpr (IsMma<Body>::value) {
      constexpr int kStages = Body::kStages;
      const int n = x0 + warp < x1 ? (x1 - x0 - warp + kWarps - 1) / kWarps : 0;
      uint8_t* ring = dyn + warp * Body::kRingBytes;
      Ahead ahead;
      // Chunk k of the warp's n: its copy, then (once its scales are there)
      // what the softmax needs of it.
      const auto start = [&](int k) {
        if ((k & 31) == 0) ahead = look_ahead(a, e, c, x0 + warp + (k + lane) * kWarps, x1);
        const int64_t at = __shfl_sync(0xffffffffu, ahead.at, k & 31);
        Body::copy(a, at, ring + (k % kStages) * Body::kStageBytes);
      };
      const auto note = [&](int k) {
        if (lane == (k & 31))
          info[warp][k % kStages] = make_float4(ahead.ks, ahead.lvs, __int_as_float(ahead.key0),
                                                __int_as_float(ahead.flags));
      };
#pragma unroll
      for (int k = 0; k < kStages; ++k) {
        if (k < n) start(k);
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
      Body::load_rows(a, p, e, c, rt, dyn);
#pragma unroll
      for (int k = 0; k < kStages; ++k)
        if (k < n) note(k);
      __syncthreads();
      body.begin(dyn);
      const int pos0 = body.rows->pos[0];  // the first row's position, the last's
      const int pos1 = body.rows->pos[min(kTile, p.rows - rt * kTile) - 1];
      const int first = pos0 - a.window + 1, last = pos1;  // slots that some row attends
      const int all0 = pos1 - a.window + 1, all1 = pos0;   // slots that every row attends
      for (int k = 0; k < n; ++k) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncwarp();
        uint8_t* stage = ring + (k % kStages) * Body::kStageBytes;
        const float4 of = info[warp][k % kStages];
        Chunk cur;
        cur.ks = of.x;
        cur.lvs = of.y;
        cur.key0 = __float_as_int(of.z);
        cur.on = __float_as_int(of.w) & 1;
        cur.window = __float_as_int(of.w) & 2;
        body.read_k(stage);
        body.scores();
        const bool edge =
            !cur.on || (cur.window && (cur.key0 < all0 || cur.key0 + kChunk - 1 > all1));
        if (a.weights) {
          if (edge)
            body.template softmax<true, true>(a, p, e, c, rt, cur);
          else
            body.template softmax<false, true>(a, p, e, c, rt, cur);
        } else if (edge) {
          body.template softmax<true, false>(a, p, e, c, rt, cur);
        } else {
          body.template softmax<false, false>(a, p, e, c, rt, cur);
        }
        body.read_v(stage);
        if (edge) body.clear_masked(cur, first, last);
        body.values();
        __syncwarp();
        if (k + kStages < n) {
          start(k + kStages);
          note(k + kStages);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
    } else {
      body.load_rows(a, p, e, c, rt, dyn);
      __syncthreads();
      body.begin(dyn);
      int x = x0 + warp;
      if (x < x1) {
        Ahead ahead = look_ahead(a, e, c, x + lane * kWarps, x1);
        int used = 0;
        for (; x < x1; x += kWarps) {
          const Chunk cur = chunk_of(ahead, used);
          body.chunk(a, p, e, c, rt, cur);
          if (++used == 32) {
            ahead = look_ahead(a, e, c, x + kWarps + lane * kWarps, x1);
            used = 0;
          }
        }
      }
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

// weights[b, c, j] += sum over the rows of KV head c of their probability of
// slot j, from the scores the attention left (4 bytes a row and slot, an
// eighth of the codes for 8 rows; computing them again would read the keys
// again, half of the codes).  A thread kSlotsT slots, 256 apart: no atomics,
// rows summed in order.  HBM bounds it: a million slots of 8 heads, 285 MB, in
// 53 us.  Not started early: waiting CTAs cost the attention 40 us there.
constexpr int kSlotsT = 4;

__global__ void __launch_bounds__(256) cache_weights_kernel(const CacheAttnArgs a) {
  extern __shared__ float2 stat[];  // of each row: its reference score, 1 / denominator
  const int rows = a.T * (a.Hq / a.c.Hkv), even = (rows + 1) & ~1;
  const int c = blockIdx.y % a.c.Hkv, b = blockIdx.y / a.c.Hkv;
  const int len = cache_len(a.s, b, a.c.block, a.status);
  const int lo = max(0, len - a.T - a.window + 1);
  wait_for_inputs();
  const int64_t u = static_cast<int64_t>(b) * a.c.Hkv + c;
  for (int r = threadIdx.x; r < rows; r += 256) stat[r] = a.row_stat[u * even + r];
  __syncthreads();
  for (int64_t j0 = static_cast<int64_t>(blockIdx.x) * 256 * kSlotsT; j0 < len;
       j0 += static_cast<int64_t>(gridDim.x) * 256 * kSlotsT) {
    const float* s = a.scores + (u * a.s.max_blocks * a.c.block + j0 + threadIdx.x) * even;
    float* to = a.weights + u * a.weights_ld + j0 + threadIdx.x;
    float sum[kSlotsT], had[kSlotsT];
    bool in[kSlotsT];
#pragma unroll
    for (int k = 0; k < kSlotsT; ++k) {
      const int64_t j = j0 + threadIdx.x + 256 * k;
      in[k] = j >= lo && j < len &&
              MSA_IN_RANGE(u * a.weights_ld + j, 1,
                           static_cast<int64_t>(a.s.batch) * a.c.Hkv * a.weights_ld, a.status);
      sum[k] = 0.f;
      had[k] = in[k] ? to[256 * k] : 0.f;
    }
    const auto add = [&](int k, float x, int r) {
      const float2 st = stat[r];
      sum[k] += x == -INFINITY ? 0.f : ex2(x - st.x) * st.y;
    };
    if ((even & 3) == 0) {
#pragma unroll 2
      for (int r = 0; r < rows; r += 4) {
        float4 x[kSlotsT];
#pragma unroll
        for (int k = 0; k < kSlotsT; ++k)
          if (in[k])
            x[k] = __ldcs(reinterpret_cast<const float4*>(
                s + static_cast<int64_t>(256 * k) * even + r));
#pragma unroll
        for (int k = 0; k < kSlotsT; ++k)
          if (in[k]) {
            add(k, x[k].x, r);
            if (r + 1 < rows) add(k, x[k].y, r + 1);
            if (r + 2 < rows) add(k, x[k].z, r + 2);
            if (r + 3 < rows) add(k, x[k].w, r + 3);
          }
      }
    } else {
      for (int r = 0; r < rows; r += 2) {
#pragma unroll
        for (int k = 0; k < kSlotsT; ++k)
          if (in[k]) {
            const float2 x = __ldcs(
                reinterpret_cast<const float2*>(s + static_cast<int64_t>(256 * k) * even + r));
            add(k, x.x, r);
            if (r + 1 < rows) add(k, x.y, r + 1);
          }
      }
    }
#pragma unroll
    for (int k = 0; k < kSlotsT; ++k)
      if (in[k]) to[256 * k] = had[k] + sum[k];
  }
}

template <int D, class Body>
cudaError_t launch_body(const CacheAttnArgs& a, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<D, Body>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, Body::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_after(cache_attn_kernel<D, Body>, dim3(a.n_ctas), kThreads, Body::kSmem, st,
                   a.sel_from_kernel != 0, a);
  if (e != cudaSuccess) return e;
  e = launch_join<D, Body::kTile>(a, st);
  if (e != cudaSuccess || !a.weights) return e;
  const int rows = a.T * (a.Hq / a.c.Hkv);  // weights: no selection
  const int64_t slots = static_cast<int64_t>(a.s.max_blocks) * a.c.block;
  const int64_t tiles = (slots + 256 * kSlotsT - 1) / (256 * kSlotsT);
  const int64_t heads = static_cast<int64_t>(a.s.batch) * a.c.Hkv;
  const dim3 grid(static_cast<unsigned>(min64(tiles, max64(1, kSms * 4 / heads))),
                  static_cast<unsigned>(heads));
  return launch_after(cache_weights_kernel, grid, 256, rows * sizeof(float2), st, false, a);
}

}  // namespace

// Tiles of 8, 16 or 32 rows: as many as the rows fill (K and V are read once
// for each tile; a tile costs the arithmetic of all its rows, held or not).
int cache_attn_tile_rows(int rows, int in_bf16) {
  return !in_bf16 || rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
}

int cache_attn_max_ctas(int tile_rows, int in_bf16) {
  return kSms * (!in_bf16         ? SimtBody<128>::kPerSm
                 : tile_rows == 8 ? MmaBody<128, 1>::kPerSm
                                  : MmaBody<128, 2>::kPerSm);
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, cudaStream_t st) {
  const int g = a.Hq / a.c.Hkv;
  const int tile = cache_attn_tile_rows(a.sel ? g : a.T * g, a.in_bf16);
  if (!a.in_bf16)
    return a.c.d == 128 ? launch_body<128, SimtBody<128>>(a, st)
                        : launch_body<64, SimtBody<64>>(a, st);
  if (tile == 8)
    return a.c.d == 128 ? launch_body<128, MmaBody<128, 1>>(a, st)
                        : launch_body<64, MmaBody<64, 1>>(a, st);
  if (tile == 16)
    return a.c.d == 128 ? launch_body<128, MmaBody<128, 2>>(a, st)
                        : launch_body<64, MmaBody<64, 2>>(a, st);
  return a.c.d == 128 ? launch_body<128, MmaBody<128, 4>>(a, st)
                      : launch_body<64, MmaBody<64, 4>>(a, st);
}

}  // namespace msa
