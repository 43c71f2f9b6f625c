// K13: norms of queries and keys for each head with the rotary position
// embedding, and their gradients.
//
// Of a row x (one token and head): z = x r w, r = (mean(x^2) + eps)^-1/2, and y
// = R z, R turning every pair of dims by the token's angles.  Backward, of g =
// R^T dy and u = w g: dx = r (u - x r^2 mean(x u)), dw = the sum over tokens
// and heads of g x r.  Everything is fp32 between one read and one rounding.
//
// Each value is read and written once, and HBM bounds a long call: 32768 tokens of
// 64 + 8 heads of 128 in bf16 take 192 us forward, 6.3 TB/s (DRAM 78 % of its peak),
// and 279 us backward, 6.5 TB/s (DRAM 83 %), with half of the issue slots.  A thread
// takes 16 values of a row, two runs of 8 half a row apart, so that both
// members of a pair are its own in either pairing; a row is d / 16 lanes.  CTAs
// take equal runs of rows of one side, whatever the tokens, with the next row's
// values under way.  The angles are the same for all heads of a token: the CTA
// computes them once for the tokens of some passes, as 64-bit integers that wrap
// around at a full turn, reduced to an eighth of a turn before they become floats.
#include "rope.cuh"

namespace msa {
namespace {

constexpr int kThreads = 256;
constexpr int kFwdPerSm = 4, kBwdPerSm = 2;  // CTAs (4: the fp32 forward spills 48 bytes a thread)
constexpr int kGroup = 8;                    // passes over which the angles are held
// Floats of the angles of a group's tokens: 8 passes of 32 rows (d = 128) or 64 are
// 2 + 256 / heads tokens and more; fewer passes a group where that does not fit.
constexpr int kAngles = 36 * 128;
// A token's angles cost a CTA about as much as the rows of this many heads.
constexpr int kTokenCost = 6;

// cos and sin (times m) of position * f / 2^64 turns.  Products wrap at whole
// turns; the nearest quarter turn is taken off as an integer, so the rest, at
// most an eighth of a turn, loses 2^-27 of a turn at most as a float.
__device__ __forceinline__ float2 turn_of(int64_t position, int64_t f, float m) {
  const uint64_t phase = static_cast<uint64_t>(position) * static_cast<uint64_t>(f);
  const uint32_t hi = static_cast<uint32_t>(phase >> 32);
  const uint32_t quarter = (hi + 0x20000000u) >> 30;
  const int rest = static_cast<int>(hi - (quarter << 30));
  float s, c;
  sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
  if (quarter & 1) {
    const float t = c;
    c = -s;
    s = t;
  }
  if (quarter & 2) {
    c = -c;
    s = -s;
  }
  return make_float2(c * m, s * m);
}

// 16 values of a row, 8 of them half a row on, as they are in memory.
template <int D, bool kBf16>
struct Raw {
  static constexpr int kWords = kBf16 ? 8 : 16;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const void* src, int64_t off) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      constexpr int kPer = kWords / 8;  // 16-byte pieces a run
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(src) +
                                                      (off + h * (D / 2)) * (kBf16 ? 2 : 4));
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint4 x = __ldcs(p + i);
        uint32_t* to = w + (h * kPer + i) * 4;
        to[0] = x.x, to[1] = x.y, to[2] = x.z, to[3] = x.w;
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // The same through shared memory, where a thread has places of its own, 16 bytes
  // in each kBytes / kPieces of a pass: it waits for its own copies only.
  static constexpr int kPieces = kWords / 4, kBytes = kPieces * kThreads * 16;
  __device__ __forceinline__ static void fetch(uint32_t to, const void* src, int64_t off) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      constexpr int kPer = kPieces / 2;
      const uint8_t* p = static_cast<const uint8_t*>(src) +
                         (off + i / kPer * (D / 2)) * (kBf16 ? 2 : 4) + i % kPer * 16;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * kThreads * 16),
                   "l"(p)
                   : "memory");
    }
  }
  __device__ __forceinline__ void read(const uint8_t* from) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint4 x = *reinterpret_cast<const uint4*>(from + i * kThreads * 16);
      w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
    }
  }
};

// The same as 8 pairs to turn, (a, b) of pair i in a[i / 2] and b[i / 2]: two
// neighbours are worked on by one packed instruction.  Of halves a run apart pair
// i is value i of both runs; of neighbours, values 2i and 2i + 1.
template <int D, bool kBf16, bool kInterleaved>
struct Pairs {
  float2 a[4], b[4];
  __device__ __forceinline__ Pairs() {}
  __device__ __forceinline__ explicit Pairs(const Raw<D, kBf16>& r) {
    float v[16];
    if constexpr (kBf16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[2 * i] = __uint_as_float(r.w[i] << 16);
        v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r.w[i]);
    }
    set(v);
  }
  __device__ __forceinline__ void set(const float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = kInterleaved ? make_float2(v[4 * i], v[4 * i + 2]) : make_float2(v[2 * i], v[2 * i + 1]);
      b[i] = kInterleaved ? make_float2(v[4 * i + 1], v[4 * i + 3])
                          : make_float2(v[8 + 2 * i], v[8 + 2 * i + 1]);
    }
  }
  __device__ __forceinline__ void get(float* v) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = kInterleaved ? 4 * i : 2 * i;
      v[x] = a[i].x;
      v[x + (kInterleaved ? 2 : 1)] = a[i].y;
      v[kInterleaved ? x + 1 : 8 + x] = b[i].x;
      v[kInterleaved ? x + 3 : 8 + x + 1] = b[i].y;
    }
  }
  // To a row's place in memory, as elements.
  __device__ __forceinline__ void store(void* dst, int64_t off) const {
    float v[16];
    get(v);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (kBf16) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 x = __floats2bfloat162_rn(v[8 * h + 2 * i], v[8 * h + 2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&x);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + off + h * (D / 2)) =
            make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(dst) + off + h * (D / 2));
        p[0] = make_float4(v[8 * h], v[8 * h + 1], v[8 * h + 2], v[8 * h + 3]);
        p[1] = make_float4(v[8 * h + 4], v[8 * h + 5], v[8 * h + 6], v[8 * h + 7]);
      }
    }
  }
  // Turns the pairs by the angles of cs (cosines, then sines), or back.
  template <bool kBack>
  __device__ __forceinline__ void turn(const float* cs, int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 c4 = *reinterpret_cast<const float4*>(cs + h * (D / 4) + lane * 4);
      const float4 s4 = *reinterpret_cast<const float4*>(cs + D / 2 + h * (D / 4) + lane * 4);
      const float2 c[2] = {make_float2(c4.x, c4.y), make_float2(c4.z, c4.w)};
      const float2 s[2] = {make_float2(s4.x, s4.y), make_float2(s4.z, s4.w)};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float2 &x = a[2 * h + k], &y = b[2 * h + k];
        const float2 minus = make_float2(-s[k].x, -s[k].y);
        const float2 u = __ffma2_rn(x, c[k], __fmul2_rn(y, kBack ? s[k] : minus));
        y = __ffma2_rn(x, kBack ? minus : s[k], __fmul2_rn(y, c[k]));
        x = u;
      }
    }
  }
};
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ float weight_at(const void* w, int bf16, int i) {
  return bf16 ? bf16_bits_to_float(static_cast<const uint16_t*>(w)[i])
              : static_cast<const float*>(w)[i];
}

// The angles of tokens t0 .. t0 + tokens: [token][cosines, sines], each in the order
// in which the lanes take them, 16 bytes side by side: the first 4 of all lanes'
// pairs, then the others.  Of halves a run apart a lane's pairs are 8 lane .. 8 lane
// + 7; of neighbours, 4 lane .. 4 lane + 3 and those d / 4 on.
// A thread computes those of one frequency.
template <int D, bool kInterleaved>
__device__ __forceinline__ void angles(const RopeArgs& a, int64_t freq, int64_t t0, int tokens,
                                       float* cs) {
  constexpr int kFreqs = D / 2;
  const int f = threadIdx.x % kFreqs;
  const int at = kInterleaved ? f : (f >> 2 & 1) * (D / 4) + (f >> 3) * 4 + (f & 3);
  for (int t = threadIdx.x / kFreqs; t < tokens; t += kThreads / kFreqs) {
    if (!MSA_IN_RANGE(t0 + t, 1, a.n, a.status)) continue;
    const float2 x = turn_of(a.positions[t0 + t], freq, a.mscale);
    cs[t * D + at] = x.x;
    cs[t * D + D / 2 + at] = x.y;
  }
}

// A CTA's rows of one side: `passes` passes over kStep rows from row0 on, a thread
// the same one of each.  Rows are counted from the first token's first.
template <int D>
struct Walk {
  static constexpr int kLanes = D / 16, kStep = kThreads / kLanes;
  int side, H, lane;
  int64_t t0;         // token of the CTA's first row
  uint32_t row, end;  // this thread's row and the end, from token t0's first
  int t, h, dt, dh;   // of `row`: token (from t0) and head; their steps
  uint32_t first;     // the CTA's first row of the pass

  // False: nothing to do.
  __device__ __forceinline__ bool begin(const RopeArgs& a) {
    side = static_cast<int>(blockIdx.x) >= a.ctas[0];
    H = a.heads[side];
    lane = threadIdx.x & (kLanes - 1);
    const int64_t all = a.n * H;
    const int ctas = a.ctas[side], cta = static_cast<int>(blockIdx.x) - (side ? a.ctas[0] : 0);
    // Whole passes, as many for each CTA as for any other but one more for the first.
    const int64_t passes = (all + kStep - 1) / kStep;
    const int64_t each = passes / ctas, more = passes - each * ctas;
    const int64_t p0 = cta * each + min64(cta, more), p1 = p0 + each + (cta < more);
    if (p0 == p1) return false;
    const int64_t r0 = p0 * kStep, r1 = min64(all, p1 * kStep);
    t0 = r0 / H;
    first = static_cast<uint32_t>(r0 - t0 * H);
    end = static_cast<uint32_t>(r1 - t0 * H);  // fits: the entry points check
    row = first + threadIdx.x / kLanes;
    t = row / H;
    h = row - t * H;
    dt = kStep / H;
    dh = kStep - dt * H;
    return true;
  }
  __device__ __forceinline__ bool in() const { return row < end; }
  __device__ __forceinline__ void next() {
    row += kStep;
    t += dt;
    h += dh;
    if (h >= H) {
      h -= H;
      ++t;
    }
  }
  // Passes whose tokens' angles are held together.
  __device__ __forceinline__ int group() const {
    return max(1, min(kGroup, (kAngles / D - 2) * H / kStep));
  }
  // Tokens of the group of `passes` passes that starts at row `from`: the first, and
  // how many.
  __device__ __forceinline__ int tokens(uint32_t from, int passes, int* token) const {
    const uint32_t to = min(end, from + static_cast<uint32_t>(passes) * kStep);
    *token = from / H;
    return static_cast<int>((to - 1) / H) - *token + 1;
  }
};

// Calls row(cs of the row's token) for every pass, the angles of a group of passes
// computed while the one before is under way.
template <int D, bool kInterleaved, typename Row>
__device__ __forceinline__ void walk_rows(const RopeArgs& a, const Walk<D>& w, float (*cs)[kAngles],
                                          Row row) {
  const int group = w.group();
  const int64_t freq = a.freqs[threadIdx.x % (D / 2)];
  int token, next_token;
  int tokens = w.tokens(w.first, group, &token);
  angles<D, kInterleaved>(a, freq, w.t0 + token, tokens, cs[0]);
  __syncthreads();
  int buffer = 0;
  for (uint32_t from = w.first; from < w.end; from += group * Walk<D>::kStep) {
    const uint32_t then = from + group * Walk<D>::kStep;
    if (then < w.end) {
      tokens = w.tokens(then, group, &next_token);
      angles<D, kInterleaved>(a, freq, w.t0 + next_token, tokens, cs[buffer ^ 1]);
    }
    for (uint32_t r = from; r < min(then, w.end); r += Walk<D>::kStep) row(cs[buffer], token);
    __syncthreads();
    buffer ^= 1;
    token = next_token;
  }
}

// The first ctas[0] CTAs take the queries' rows, the others the keys'.
template <int D, bool kBf16, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kFwdPerSm) norm_rope_kernel(const RopeArgs a) {
  __shared__ __align__(16) float cs[2][kAngles];
  Walk<D> w;
  if (!w.begin(a)) return;
  const int lane = w.lane, H = w.H;
  const void* src = a.x[w.side];
  const int64_t stride = a.stride[w.side];
  const bool norm = a.weight[w.side] != nullptr;
  Pairs<D, kBf16, kInterleaved> weight;
  {
    float v[16];
#pragma unroll
    for (int k = 0; k < 16; ++k)
      v[k] = norm ? weight_at(a.weight[w.side], a.w_bf16, (k >> 3) * (D / 2) + lane * 8 + (k & 7))
                  : 1.f;
    weight.set(v);
  }
  // A row's values come in while the one before is worked on.
  Raw<D, kBf16> ahead;
  const auto load = [&](const Walk<D>& at) {
    const int64_t from = (at.t0 + at.t) * stride + at.h * D + lane * 8;
    if (at.in() && MSA_IN_RANGE(from, D / 2 + 8, (a.n - 1) * stride + H * D, a.status))
      ahead.load(src, from);
    else
      ahead.clear();
  };
  load(w);
  walk_rows<D, kInterleaved>(a, w, cs, [&](const float* c, int token) {
    const Walk<D> at = w;
    Pairs<D, kBf16, kInterleaved> x(ahead);
    w.next();
    load(w);
    if (norm) {
      float2 ss = both(0.f);
#pragma unroll
      for (int k = 0; k < 4; ++k) ss = __ffma2_rn(x.a[k], x.a[k], __ffma2_rn(x.b[k], x.b[k], ss));
      const float2 r = both(
          rsqrtf(row_sum<Walk<D>::kLanes>(ss.x + ss.y) * (1.f / D) + a.eps));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x.a[k] = __fmul2_rn(__fmul2_rn(x.a[k], r), weight.a[k]);
        x.b[k] = __fmul2_rn(__fmul2_rn(x.b[k], r), weight.b[k]);
      }
    }
    if (!at.in()) return;
    x.template turn<false>(c + (at.t - token) * D, lane);
    const int64_t to = ((at.t0 + at.t) * H + at.h) * D + lane * 8;
    if (MSA_IN_RANGE(to, D / 2 + 8, a.n * H * D, a.status)) x.store(a.out[w.side], to);
  });
}

// A sum in two floats: lo takes what an addition to hi rounds off (Knuth's
// two-sum), so that a sum of any length keeps fp32's bits.  (In 64 bits, at the 1.25
// TFLOP/s that a GB300 is given, the last kernel's additions alone would take some 2 us
// of the 2K-token step's 11.)
struct Sum {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {
    const float s = hi + x, b = s - hi;
    lo += (hi - (s - b)) + (x - b);
    hi = s;
  }
  __device__ __forceinline__ void add(const Sum& x) {
    add(x.hi);
    lo += x.lo;
  }
  __device__ __forceinline__ float value() const {  // hi infinite: lo is a NaN
    return fabsf(hi) < INFINITY ? hi + lo : hi;
  }
};

// A thread's sums of the weights' gradients: kSumPasses passes in registers, then
// over the warp's lanes of the same dims, each of which gets kOwn of the 16 values to
// add to sums of its own in shared memory: [hi, lo][thread][kOwn].
constexpr int kSumPasses = 8;
template <int D>
struct Columns {
  static constexpr int kLanes = D / 16, kOwn = 16 * kLanes / 32;
  static constexpr int kBytes = 2 * kThreads * kOwn * static_cast<int>(sizeof(float));
  __device__ __forceinline__ static float* at(float* sums, int half, int thread) {
    return sums + (half * kThreads + thread) * kOwn;
  }
  __device__ __forceinline__ static void clear(float* sums) {
#pragma unroll
    for (int k = 0; k < kOwn; ++k)
      at(sums, 0, threadIdx.x)[k] = at(sums, 1, threadIdx.x)[k] = 0.f;
  }
  __device__ __forceinline__ static void add(float* sums, float* v) {
#pragma unroll
    for (int o = 16, n = 8; o >= kLanes; o >>= 1, n >>= 1) {
      const bool up = threadIdx.x & o;
#pragma unroll
      for (int k = 0; k < n; ++k) {
        const float give = up ? v[k] : v[n + k], keep = up ? v[n + k] : v[k];
        v[k] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
    float *hi = at(sums, 0, threadIdx.x), *lo = at(sums, 1, threadIdx.x);
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      Sum s{hi[k], lo[k]};
      s.add(v[k]);
      hi[k] = s.hi;
      lo[k] = s.lo;
    }
  }
  // Column `dim` of all warps.
  __device__ __forceinline__ static Sum column(float* sums, int dim) {
    const int k = dim / (D / 2) * 8 + (dim & 7);  // the value among a lane's 16
    int lane = dim % (D / 2) / 8;
#pragma unroll
    for (int o = 16, n = 8; o >= kLanes; o >>= 1, n >>= 1) lane |= k & n ? o : 0;
    Sum s{0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const int thread = 32 * w + lane;
      s.add(Sum{at(sums, 0, thread)[k % kOwn], at(sums, 1, thread)[k % kOwn]});
    }
    return s;
  }
};

// The gradients' kernel has two inputs: bf16 values come through a ring in shared
// memory, kDepth passes under way.  fp32 ones, which are twice the bytes a pass,
// come in registers, one pass ahead, as the forward's do (32K tokens of 32 + 4 heads
// of 128 in fp32: 455 us through the ring, 287 in registers; the bf16 forward of 64
// + 8 heads 241 and 191).
template <int D, bool kBf16>
struct Ring {
  using R = Raw<D, kBf16>;
  static constexpr int kDepth = kBf16 ? 3 : 1;
  static constexpr int kPass = kBf16 ? 2 * R::kBytes : 0;
  static constexpr int kSums = static_cast<int>(2 * kAngles * sizeof(float));  // from here on
  static constexpr int kRing = kSums + Columns<D>::kBytes;
  static constexpr int kSmem = kRing + kDepth * kPass;
};
template <int D, bool kBf16, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kBwdPerSm) norm_rope_bwd_kernel(const RopeArgs a) {
  using R = Raw<D, kBf16>;
  constexpr int kDepth = Ring<D, kBf16>::kDepth, kPass = Ring<D, kBf16>::kPass;
  extern __shared__ __align__(16) uint8_t dyn[];  // the angles, the weights' sums, the ring
  float(*cs)[kAngles] = reinterpret_cast<float(*)[kAngles]>(dyn);
  float* sums = reinterpret_cast<float*>(dyn + Ring<D, kBf16>::kSums);
  uint8_t* mine = dyn + Ring<D, kBf16>::kRing + threadIdx.x * 16;
  const uint32_t place = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
  Walk<D> w;
  let_next_start();
  if (!w.begin(a)) {  // its sums are read
    if (a.weight[w.side] && threadIdx.x < D)
      a.part[static_cast<int64_t>(blockIdx.x) * D + threadIdx.x] = make_float2(0.f, 0.f);
    return;
  }
  const int lane = w.lane, H = w.H;
  const bool norm = a.weight[w.side] != nullptr;
  const void *src = a.x[w.side], *grad = a.dy[w.side];
  const int64_t stride = a.stride[w.side], dy_stride = a.dy_stride[w.side];
  Pairs<D, kBf16, kInterleaved> weight, dw;
  {
    float v[16];
#pragma unroll
    for (int k = 0; k < 16; ++k)
      v[k] = norm ? weight_at(a.weight[w.side], a.w_bf16, (k >> 3) * (D / 2) + lane * 8 + (k & 7))
                  : 1.f;
    weight.set(v);
  }
  int summed = 0;  // passes in dw
  const auto sum_up = [&] {
    float v[16];
    dw.get(v);
    Columns<D>::add(sums, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) dw.a[k] = dw.b[k] = both(0.f);
    summed = 0;
  };
#pragma unroll
  for (int k = 0; k < 4; ++k) dw.a[k] = dw.b[k] = both(0.f);
  if (norm) Columns<D>::clear(sums);
  Walk<D> ahead = w;
  R next_g, next_x;  // fp32
  const auto fetch = [&](int slot) {
    if constexpr (!kBf16) {
      next_g.clear();
      next_x.clear();
    }
    if (ahead.in()) {
      const int64_t t = ahead.t0 + ahead.t, h = ahead.h * D + lane * 8;
      const bool g_in = MSA_IN_RANGE(t * dy_stride + h, D / 2 + 8,
                                     (a.n - 1) * dy_stride + H * D, a.status);
      const bool x_in = norm && MSA_IN_RANGE(t * stride + h, D / 2 + 8,
                                             (a.n - 1) * stride + H * D, a.status);
      if constexpr (kBf16) {
        if (g_in) R::fetch(place + slot * kPass, grad, t * dy_stride + h);
        if (x_in) R::fetch(place + slot * kPass + R::kBytes, src, t * stride + h);
      } else {
        if (g_in) next_g.load(grad, t * dy_stride + h);
        if (x_in) next_x.load(src, t * stride + h);
      }
    }
    ahead.next();
    if constexpr (kBf16) asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int k = 0; k < kDepth; ++k) fetch(k);
  int slot = 0;
  walk_rows<D, kInterleaved>(a, w, cs, [&](const float* c, int token) {
    const Walk<D> at = w;
    R raw_g, raw_x;
    if constexpr (kBf16) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
      raw_g.clear();
      raw_x.clear();
      if (at.in()) {
        raw_g.read(mine + slot * kPass);
        if (norm) raw_x.read(mine + slot * kPass + R::kBytes);
      }
    } else {
      raw_g = next_g;
      raw_x = next_x;
      fetch(0);
    }
    Pairs<D, kBf16, kInterleaved> g(raw_g), x(raw_x);
    w.next();
    g.template turn<true>(c + (at.in() ? at.t - token : 0) * D, lane);
    if (norm) {
      float2 ss = both(0.f), xu = both(0.f), u[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        u[k] = __fmul2_rn(weight.a[k], g.a[k]);
        u[4 + k] = __fmul2_rn(weight.b[k], g.b[k]);
        ss = __ffma2_rn(x.a[k], x.a[k], __ffma2_rn(x.b[k], x.b[k], ss));
        xu = __ffma2_rn(x.a[k], u[k], __ffma2_rn(x.b[k], u[4 + k], xu));
      }
      const float r = rsqrtf(row_sum<Walk<D>::kLanes>(ss.x + ss.y) * (1.f / D) + a.eps);
      // Rows past the end are zeros: they add none to dw, unless r is infinite.
      const float rw = at.in() ? r : 0.f;
      // r times the mean first: r^2 alone passes fp32's range for rows below 2^-64.
      const float f = -r * (r * (row_sum<Walk<D>::kLanes>(xu.x + xu.y) * (1.f / D)));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        dw.a[k] = __ffma2_rn(g.a[k], __fmul2_rn(x.a[k], both(rw)), dw.a[k]);
        dw.b[k] = __ffma2_rn(g.b[k], __fmul2_rn(x.b[k], both(rw)), dw.b[k]);
        g.a[k] = __fmul2_rn(both(r), __ffma2_rn(x.a[k], both(f), u[k]));
        g.b[k] = __fmul2_rn(both(r), __ffma2_rn(x.b[k], both(f), u[4 + k]));
      }
      if (++summed == kSumPasses) sum_up();
    }
    const int64_t to = ((at.t0 + at.t) * H + at.h) * D + lane * 8;
    if (at.in() && MSA_IN_RANGE(to, D / 2 + 8, a.n * H * D, a.status)) g.store(a.out[w.side], to);
    if constexpr (kBf16) {
      fetch(slot);
      slot = slot + 1 == kDepth ? 0 : slot + 1;
    }
  });
  if (!norm) return;
  if (summed) sum_up();
  __syncthreads();
  if (threadIdx.x < D) {
    const Sum sum = Columns<D>::column(sums, threadIdx.x);
    a.part[static_cast<int64_t>(blockIdx.x) * D + threadIdx.x] = make_float2(sum.hi, sum.lo);
  }
}

// The weights' gradients from the CTAs' sums: blockIdx.x the side, a thread a
// column of every kSlices-th CTA.
constexpr int kSlices = 8;
template <int D>
__global__ void __launch_bounds__(D * kSlices) norm_rope_dw_kernel(const RopeArgs a) {
  __shared__ Sum sums[kSlices][D];
  const int side = blockIdx.x, k = threadIdx.x % D, slice = threadIdx.x / D;
  wait_for_inputs();
  if (!a.dweight[side]) return;
  const float2* part = a.part + (side ? static_cast<int64_t>(a.ctas[0]) * D : 0) + k;
  Sum sum{0.f, 0.f};
  if (a.n > 0) {
#pragma unroll 8
    for (int c = slice; c < a.ctas[side]; c += kSlices) {
      const float2 x = part[static_cast<int64_t>(c) * D];
      sum.add(Sum{x.x, x.y});
    }
  }
  sums[slice][k] = sum;
  __syncthreads();
  if (slice) return;
#pragma unroll
  for (int i = 1; i < kSlices; ++i) sum.add(sums[i][k]);
  if (a.w_bf16)
    static_cast<__nv_bfloat16*>(a.dweight[side])[k] = __float2bfloat16_rn(sum.value());
  else
    static_cast<float*>(a.dweight[side])[k] = sum.value();
}

// CTAs of the two sides: at most `all`, shared by what their rows and angles cost
// (with 64 + 8 heads by rows alone, the keys' CTAs ended last: 423 us for 276),
// none without a pass, and each side that has rows at least one.
void split_ctas(int64_t n, const int* heads, int d, int64_t all, int* ctas) {
  const int step = kThreads / (d / 16);
  const int64_t q = (n * heads[0] + step - 1) / step, k = (n * heads[1] + step - 1) / step;
  if (q + k > all) {
    const int64_t wq = heads[0] + kTokenCost, wk = heads[1] + kTokenCost;
    const int64_t share = min64(all - 1, (all * wk + (wq + wk) / 2) / (wq + wk));
    ctas[1] = k ? static_cast<int>(max64(1, min64(k, share))) : 0;
    ctas[0] = static_cast<int>(min64(q, all - ctas[1]));
  } else {
    ctas[0] = static_cast<int>(max64(1, q));
    ctas[1] = static_cast<int>(k);
  }
}

template <int D, bool kBf16, bool kInterleaved>
cudaError_t launch_bwd(const RopeArgs& a, cudaStream_t st) {
  constexpr int kSmem = Ring<D, kBf16>::kSmem;
  const cudaError_t e = cudaFuncSetAttribute(norm_rope_bwd_kernel<D, kBf16, kInterleaved>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(a.ctas[0] + a.ctas[1]));
  return launch_after(norm_rope_bwd_kernel<D, kBf16, kInterleaved>, grid, kThreads, kSmem, st, false,
                      a);
}

}  // namespace

cudaError_t launch_norm_rope(const RopeArgs& a0, cudaStream_t st) {
  RopeArgs a = a0;
  split_ctas(a.n, a.heads, a.d, kSms * kFwdPerSm, a.ctas);
  const dim3 grid(static_cast<unsigned>(a.ctas[0] + a.ctas[1]));
  void (*kernel)(RopeArgs);
  if (a.d == 128)
    kernel = a.bf16 ? (a.interleaved ? norm_rope_kernel<128, true, true>
                                     : norm_rope_kernel<128, true, false>)
                    : (a.interleaved ? norm_rope_kernel<128, false, true>
                                     : norm_rope_kernel<128, false, false>);
  else
    kernel = a.bf16 ? (a.interleaved ? norm_rope_kernel<64, true, true>
                                     : norm_rope_kernel<64, true, false>)
                    : (a.interleaved ? norm_rope_kernel<64, false, true>
                                     : norm_rope_kernel<64, false, false>);
  return launch_after(kernel, grid, kThreads, 0, st, false, a);
}

void norm_rope_bwd_ctas(int64_t n, const int* heads, int d, int* ctas) {
  split_ctas(n, heads, d, kSms * kBwdPerSm, ctas);
}

cudaError_t launch_norm_rope_bwd(const RopeArgs& a, cudaStream_t st) {
  if (a.n > 0) {
    cudaError_t e;
    if (a.d == 128)
      e = a.bf16 ? (a.interleaved ? launch_bwd<128, true, true>(a, st)
                                  : launch_bwd<128, true, false>(a, st))
                 : (a.interleaved ? launch_bwd<128, false, true>(a, st)
                                  : launch_bwd<128, false, false>(a, st));
    else
      e = a.bf16 ? (a.interleaved ? launch_bwd<64, true, true>(a, st)
                                  : launch_bwd<64, true, false>(a, st))
                 : (a.interleaved ? launch_bwd<64, false, true>(a, st)
                                  : launch_bwd<64, false, false>(a, st));
    if (e != cudaSuccess) return e;
  }
  if (!a.weight[0] && !a.weight[1]) return cudaSuccess;
  return launch_after(a.d == 128 ? norm_rope_dw_kernel<128> : norm_rope_dw_kernel<64>, dim3(2),
                      a.d * kSlices, 0, st, a.n > 0, a);
}

}  // namespace msa
