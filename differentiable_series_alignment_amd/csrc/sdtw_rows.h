// Device helpers of the token losses (sdtw_tokens.hip, sdtw_distill.hip): one
// pass over rows of logits in fp32, bf16 or fp16 with a running maximum and
// sums, block reductions, and the selection of a row's largest entries.
#pragma once
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "sdtw.h"
#include "sdtw_device.h"

namespace sdtw {

// A row, or a part of one, belongs to a team of NT threads: one wave (64,
// four teams to a block), a block of 256, or one of 512.
template <int NT> constexpr int kTeamBlock = NT < 256 ? 256 : NT;
template <int NT> constexpr int kTeams = kTeamBlock<NT> / NT;
template <int NT> __device__ __forceinline__ uint32_t team_tid() {
  return NT < 256 ? threadIdx.x % NT : threadIdx.x;
}
template <int NT> __device__ __forceinline__ uint32_t team_id() {
  return NT < 256 ? threadIdx.x / NT : 0;
}
// Orders the team's LDS and memory accesses before against those behind it.
template <int NT> __device__ __forceinline__ void team_sync() {
  if (NT == kWave) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  } else {
    __syncthreads();
  }
}

// Logits element types: `Raw` is a 16-byte vector of them.
template <typename E> struct RowType;
template <> struct RowType<float> {
  typedef float Raw __attribute__((ext_vector_type(4)));
  typedef float Wide __attribute__((ext_vector_type(4)));
};
template <> struct RowType<__bf16> {
  typedef __bf16 Raw __attribute__((ext_vector_type(8)));
  typedef float Wide __attribute__((ext_vector_type(8)));
};
template <> struct RowType<_Float16> {
  typedef _Float16 Raw __attribute__((ext_vector_type(8)));
  typedef float Wide __attribute__((ext_vector_type(8)));
};
template <typename E> constexpr int kRowVec = 16 / (int)sizeof(E);
// Vectors a thread requests together (a group), and entries of them.
template <typename E> constexpr int kRowUnroll = 4;
template <typename E> constexpr int kGroup = kRowUnroll<E> * kRowVec<E>;

// 16 bytes of a row, at the elements' own alignment (rows of an odd length
// start anywhere).  ONCE: past the caches (see read_once; a template argument
// because a branch on a variable ends as one ordinary access).
template <typename E> struct RowUnaligned {
  typedef typename RowType<E>::Raw T __attribute__((aligned(alignof(E)), may_alias));
};
template <typename E, bool ONCE = false>
__device__ __forceinline__ typename RowType<E>::Raw row_load(const E* p) {
  typedef typename RowUnaligned<E>::T U;
  return ONCE ? __builtin_nontemporal_load(reinterpret_cast<const U*>(p))
              : *reinterpret_cast<const U*>(p);
}
template <typename E, bool ONCE = false>
__device__ __forceinline__ void row_store(E* p, typename RowType<E>::Wide x) {
  typedef typename RowUnaligned<E>::T U;
  const auto v = __builtin_convertvector(x, typename RowType<E>::Raw);   // rounds to nearest even
  if (ONCE) __builtin_nontemporal_store(v, reinterpret_cast<U*>(p));
  else *reinterpret_cast<U*>(p) = v;
}
template <typename E>
__device__ __forceinline__ typename RowType<E>::Wide row_wide(typename RowType<E>::Raw v) {
  return __builtin_convertvector(v, typename RowType<E>::Wide);
}

// The rows of a call: row r of `rows` is (r / n, r % n) of the caller's two
// leading dimensions, ld0 and ld1 elements apart.
struct RowsIn {
  const void* z;
  int64_t ld0, ld1;
  uint32_t rows, n;
  uint32_t V;
};
template <typename E> __device__ __forceinline__ const E* row_ptr(const RowsIn& a, uint32_t r) {
  const uint32_t q = a.n >= a.rows ? 0 : r / a.n;
  return static_cast<const E*>(a.z) + (int64_t)q * a.ld0 + (int64_t)(r - q * a.n) * a.ld1;
}
// Entries z[0, len) of a row, from the row's entry lo on: whole vectors start
// `head` entries in, on 16 bytes of memory (rows of an odd length start
// anywhere: reading 1024 of 65537 fp16 entries took 33.6 us with vectors from
// the first entry on, where 1024 of 65536 took 27.5).
template <typename E> struct Part {
  const E* z;
  uint32_t lo, len, head, nvec;
  // The entry before or behind the vectors that thread tid has (>= len: none).
  __device__ __forceinline__ uint32_t rest(uint32_t tid) const {
    return tid < head ? tid : tid + nvec * kRowVec<E>;
  }
  __device__ __forceinline__ uint32_t rests() const { return len - nvec * kRowVec<E>; }
  __device__ __forceinline__ const E* vectors() const { return z + head; }
  // Bit of entry i in a bitmap in which a vector's bits are in one word.
  __device__ __forceinline__ uint32_t bit(uint32_t i) const {
    return i + (kRowVec<E> - head) % kRowVec<E>;
  }
};
// `aligned`: the address that the vectors are aligned by (the entries', or
// those that are written).
template <typename E>
__device__ __forceinline__ Part<E> make_part(const E* row, uint32_t lo, uint32_t hi,
                                             const void* aligned) {
  constexpr uint32_t n = kRowVec<E>;
  const uint32_t off = ((uint32_t)(uintptr_t)aligned & 15u) / (uint32_t)sizeof(E);
  Part<E> p{row + lo, lo, hi - lo, (n - off) % n, 0};
  p.head = min(p.head, p.len);
  p.nvec = (p.len - p.head) / n;
  return p;
}
// 32-bit words of a part's bitmap.
template <typename E> __host__ __device__ inline uint32_t bitmap_words(uint32_t len) {
  return (len + kRowVec<E> + 31) / 32;
}
// An integer array that goes with the rows (tokens, lists of ids), 4 or 8
// bytes an element.
struct IdsIn {
  const void* p;
  int64_t ld0, ld1;
  int bytes;
};
__device__ __forceinline__ int64_t id_load(const IdsIn& t, uint32_t rows, uint32_t n, uint32_t r,
                                           uint32_t k) {
  const uint32_t q = n >= rows ? 0 : r / n;
  const int64_t i = (int64_t)q * t.ld0 + (int64_t)(r - q * n) * t.ld1 + k;
  return t.bytes == 8 ? static_cast<const int64_t*>(t.p)[i]
                      : (int64_t) static_cast<const int32_t*>(t.p)[i];
}

// Exponents.  With c = log2(e) / temperature (rounded once to fp32: a
// temperature off by 2^-24, the same for every use of it) the exponent of an
// entry against a reference is t = z c - ref, one fma, exact up to its own
// rounding whatever ref is; ref is the running maximum times c, at least
// -kFar, so that a part with nothing above -inf (or the lowest value) has
// exponents of -inf and no NaN.  Rows whose maximum is beyond kFar / c in
// size ("far": logits of 1e8 and more, rows of the type's lowest value alone)
// would lose the difference to the rounding of ref; they take t = (z - max) c.
constexpr float kFar = 0x1p28f;
struct Exponent {
  float c, ref;
  bool far;
};
template <bool FAR> __device__ __forceinline__ float exponent(const Exponent& x, float z) {
  return FAR ? (z - x.ref) * x.c : __builtin_fmaf(z, x.c, -x.ref);
}
__device__ __forceinline__ float reference(float m, float c) { return fmaxf(m * c, -kFar); }
// The same in fp64, for the few entries whose logarithm is wanted.
__device__ __forceinline__ double exponent64(const Exponent& x, float z) {
  return x.far ? ((double)z - (double)x.ref) * (double)x.c
               : (double)z * (double)x.c - (double)x.ref;
}

// Statistics of a part of a row: m its maximum, and over its entries, with t
// their exponents,  s = sum 2^t,  w = sum 2^t t.  Sums of one group are fp32,
// everything longer fp64: log s then carries no more than the rounding of the
// single terms.
struct RowSums {
  float m;
  double s, w;
};

// To the reference of another maximum (2^(t + d) (t + d) summed: f (w + d s)).
template <bool W> __device__ __forceinline__ void sums_move(RowSums& r, float c, float m) {
  const float d = reference(r.m, c) - reference(m, c);
  const double f = (double)hw_exp2(d);
  if (W) r.w = f * (r.w + (double)d * r.s);
  r.s *= f;
  r.m = m;
}

template <typename E> __device__ __forceinline__ float wide_max(typename RowType<E>::Wide x) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < kRowVec<E>; ++i) m = fmaxf(m, x[i]);
  return m;
}

// A team's share of memory for one row.
template <typename E> struct Group {
  typename RowType<E>::Raw v[kRowUnroll<E>];
};
// Vectors base + u NT + tid of a part of nvec >= 1 (the last one again in the
// place of those behind it: no branch, whose two sides would have to agree on
// how many loads are under way).
template <typename E, int NT, bool ONCE = false>
__device__ __forceinline__ Group<E> group_load(const E* p, uint32_t base, uint32_t nvec) {
  constexpr int U = kRowUnroll<E>, n = kRowVec<E>;
  Group<E> g;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t v = min(base + u * NT + team_tid<NT>(), nvec - 1);
    g.v[u] = row_load<E, ONCE>(p + (size_t)v * n);
  }
  return g;
}
// The same with -inf in the place of those behind the last.
template <typename E, int NT>
__device__ __forceinline__ Group<E> group_cut(Group<E> g, uint32_t base, uint32_t nvec) {
  if (base + kRowUnroll<E> * NT > nvec) {
#pragma unroll
    for (int u = 0; u < kRowUnroll<E>; ++u)
      if (base + u * NT + team_tid<NT>() >= nvec)
        g.v[u] = (typename RowType<E>::Raw)(E)-__builtin_inff();
  }
  return g;
}
template <typename E> __device__ __forceinline__ float group_max(const Group<E>& g) {
  float m = wide_max<E>(row_wide<E>(g.v[0]));
#pragma unroll
  for (int u = 1; u < kRowUnroll<E>; ++u) m = fmaxf(m, wide_max<E>(row_wide<E>(g.v[u])));
  return m;
}

// Adds entry z to fp32 sums.
template <bool W, bool FAR>
__device__ __forceinline__ void term_add(const Exponent& x, float z, float& s, float& w) {
  const float t = exponent<FAR>(x, z);
  const float e = hw_exp2(t);
  s += e;
  if (W) w = __builtin_fmaf(e, fmaxf(t, -200.f), w);   // 0 * -inf is no NaN
}

// Adds a group.
template <typename E, bool W>
__device__ __forceinline__ void group_add(RowSums& r, const Exponent& x, const Group<E>& g) {
  constexpr int U = kRowUnroll<E>, n = kRowVec<E>;
  float s = 0.f, w = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const auto z = row_wide<E>(g.v[u]);
    float su = 0.f, wu = 0.f;
#pragma unroll
    for (int i = 0; i < n; ++i) term_add<W, false>(x, z[i], su, wu);
    s += su;
    if (W) w += wu;
  }
  r.s += (double)s;
  if (W) r.w += (double)w;
}

// Bits of the bitmap `listed` (one for each entry of a part) for vector v.
template <typename E>
__device__ __forceinline__ unsigned listed_bits(const uint32_t* listed, const Part<E>& p,
                                                uint32_t v) {
  constexpr int n = kRowVec<E>;
  const uint32_t at = v + p.bit(p.head) / n;       // (a multiple of n)
  const unsigned byte = reinterpret_cast<const uint8_t*>(listed)[at * n / 8];
  return n == 8 ? byte : byte >> (at % 2 * 4) & 15u;
}
template <typename E>
__device__ __forceinline__ bool is_listed(const uint32_t* listed, const Part<E>& p, uint32_t i) {
  const uint32_t bit = p.bit(i);
  return listed[bit >> 5] >> (bit & 31) & 1u;
}
// Entry i of a vector to -inf where bit i of `out` is set.
template <typename E>
__device__ __forceinline__ typename RowType<E>::Raw vector_leave(typename RowType<E>::Raw v,
                                                                 unsigned out) {
  typedef unsigned Words __attribute__((ext_vector_type(4)));
  constexpr unsigned none = sizeof(E) == 4                    ? 0xFF800000u
                            : std::is_same<E, __bf16>::value  ? 0xFF80FF80u
                                                              : 0xFC00FC00u;
  Words w = __builtin_bit_cast(Words, v);
  auto bit = [&](int i) { return (unsigned)((int)(out << (31 - i)) >> 31); };
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const unsigned m = sizeof(E) == 4 ? bit(k)
                                      : (bit(2 * k) & 0xFFFFu) | (bit(2 * k + 1) & ~0xFFFFu);
    w[k] = (none & m) | (w[k] & ~m);
  }
  return __builtin_bit_cast(typename RowType<E>::Raw, w);
}
// A group from vector `base` on without its listed entries (-inf in their
// place), few of them: a wave changes a vector where any of its lanes has one
// (selects for all cost two to four operations an entry beside its fma,
// exponential and sum: 53 us for 2048 rows of 50016 bf16 entries, 46 so).
template <typename E, int NT>
__device__ __forceinline__ void group_leave(Group<E>& g, uint32_t base, const uint32_t* listed,
                                            const Part<E>& p) {
  constexpr int U = kRowUnroll<E>;
  unsigned out[U];
  // (Behind the last vector there are none, whatever the bits.)
#pragma unroll
  for (int u = 0; u < U; ++u)
    out[u] = listed_bits<E>(listed, p, min(base + u * NT + team_tid<NT>(), p.nvec - 1));
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (__builtin_amdgcn_ballot_w64(out[u] != 0) != 0) g.v[u] = vector_leave<E>(g.v[u], out[u]);
}

// A part's first groups, requested before anything else is done for the row:
// HG of them that stay in registers, and the two behind them (ALL: there are
// none).
template <typename E, int HG> struct RowStart {
  Group<E> held[HG ? HG : 1];        // (HG == 0: unused)
  Group<E> a, b;
};
template <typename E, int NT, bool ONCE, int HG, bool ALL>
__device__ __forceinline__ RowStart<E, HG> row_start(const Part<E>& part) {
  constexpr int step = kRowUnroll<E> * NT;
  RowStart<E, HG> s;
  if (part.nvec == 0) return s;
#pragma unroll
  for (int h = 0; h < HG; ++h)
    s.held[h] = group_load<E, NT, ONCE>(part.vectors(), h * step, part.nvec);
  if (!ALL) {
    s.a = group_load<E, NT, ONCE>(part.vectors(), HG * step, part.nvec);
    s.b = group_load<E, NT, ONCE>(part.vectors(), (HG + 1) * step, part.nvec);
  }
  return s;
}
// f(group, base) for every group of a part from vector `base` on, of which a
// and b are the first two: two groups are always on their way, one of them
// while the other is used.
template <typename E, int NT, bool ONCE, typename F>
__device__ __forceinline__ void each_group(const E* p, uint32_t base, uint32_t nvec, Group<E>& a,
                                           Group<E>& b, F f) {
  constexpr int step = kRowUnroll<E> * NT;
  if (base >= nvec) return;
  for (;;) {
    f(a, base);
    a = group_load<E, NT, ONCE>(p, base + 2 * step, nvec);
    __builtin_amdgcn_sched_barrier(0);
    if (base + step >= nvec) break;
    f(b, base + step);
    b = group_load<E, NT, ONCE>(p, base + 3 * step, nvec);
    __builtin_amdgcn_sched_barrier(0);
    base += 2 * step;
    if (base >= nvec) break;
  }
}

// A part of a row by a team: group g holds vectors [g U NT, (g + 1) U NT) of
// the part; the entries before and behind the vectors belong to threads 0, 1,
// ...  With LISTED the entries in the bitmap stay out of the sums and of the
// maximum.  gmax, if not null, gets the maximum of each thread's groups,
// [groups][NT].  `start`: what row_start requested; its held groups stay
// (listed entries as -inf).
template <typename E, int NT, bool W, bool LISTED, bool ONCE, int HG, bool ALL>
__device__ __forceinline__ RowSums row_sums(const Part<E>& part, float c, const uint32_t* listed,
                                            float* gmax, RowStart<E, HG>& start) {
  static_assert(!(W && LISTED), "a list leaves entries out of s alone");
  constexpr int step = kRowUnroll<E> * NT;
  const uint32_t nvec = part.nvec, tid = team_tid<NT>();
  const E* p = part.vectors();
  RowSums r{-__builtin_inff(), 0.0, 0.0};
  auto add = [&](Group<E>& g, uint32_t base) {
    g = group_cut<E, NT>(g, base, nvec);
    if (LISTED) group_leave<E, NT>(g, base, listed, part);
    const float m = group_max<E>(g);
    if (gmax) gmax[base / kRowUnroll<E> + tid] = m;
    if (m > r.m) sums_move<W>(r, c, m);
    const Exponent x{c, reference(r.m, c), false};
    // With groups held, or a list, registers are short: the entries are
    // converted once more rather than kept from the maximum on.
    Group<E> again = g;
    if (sizeof(E) == 2 && (HG > 1 || LISTED))
#pragma unroll
      for (int u = 0; u < kRowUnroll<E>; ++u) asm volatile("" : "+v"(again.v[u]));
    group_add<E, W>(r, x, again);
  };
#pragma unroll
  for (int h = 0; h < HG; ++h)
    if (h * step < nvec) add(start.held[h], h * step);
  if (!ALL) each_group<E, NT, ONCE>(p, HG * step, nvec, start.a, start.b, add);
  const uint32_t rest = part.rest(tid);
  if (rest < part.len && !(LISTED && is_listed<E>(listed, part, rest))) {
    const float v = (float)part.z[rest];
    if (v > r.m) sums_move<W>(r, c, v);
    float s = 0.f, w = 0.f;
    term_add<W, false>(Exponent{c, reference(r.m, c), false}, v, s, w);
    r.s += (double)s;
    if (W) r.w += (double)w;
  }
  return r;
}
// The same for a far row, whose maximum is known.  (Inlined: a call, though
// hardly ever made, keeps the part in memory for every row; 2048 rows of 50016
// bf16 entries with a list took 50 us so, 44 inlined.)
template <typename E, int NT, bool W, bool LISTED>
__device__ __forceinline__ RowSums row_sums_far(const Part<E>& part, float c, float m,
                                                const uint32_t* listed) {
  RowSums r{m, 0.0, 0.0};
  for (uint32_t i = team_tid<NT>(); i < part.len; i += NT)
    if (!(LISTED && is_listed<E>(listed, part, i))) {
      float s = 0.f, w = 0.f;
      term_add<W, true>(Exponent{c, m, true}, (float)part.z[i], s, w);
      r.s += (double)s;
      if (W) r.w += (double)w;
    }
  return r;
}
__device__ __forceinline__ bool far_row(float m, float c) {
  return m != -__builtin_inff() && !(fabsf(m * c) < kFar);
}
__device__ __forceinline__ Exponent row_exponent(float m, float c) {
  const bool far = far_row(m, c);
  return Exponent{c, far ? m : reference(m, c), far};
}

// The reference of a row, or part, of maximum m in fp64, far or not.
__device__ __forceinline__ double reference64(float m, float c) {
  return far_row(m, c) ? (double)m * (double)c : (double)reference(m, c);
}
// 2^d for d <= 0 to 1e-11 relative, by the exponential's series of nine terms
// behind the constant one on |x| <= ln2 / 2 (what is left out: x^10 / 10!).  It
// weighs a whole sum, whose own error averages over its terms: fp32's 6e-8 there
// would be most of the error of a loss near zero.
__device__ __forceinline__ double exp2_wide(double d) {
  d = fmin(fmax(d, -2000.0), 0.0);
  const double n = rint(d), x = (d - n) * kLn2;
  double r = 1.0 / 362880;
  r = __builtin_fma(r, x, 1.0 / 40320);
  r = __builtin_fma(r, x, 1.0 / 5040);
  r = __builtin_fma(r, x, 1.0 / 720);
  r = __builtin_fma(r, x, 1.0 / 120);
  r = __builtin_fma(r, x, 1.0 / 24);
  r = __builtin_fma(r, x, 1.0 / 6);
  r = __builtin_fma(r, x, 0.5);
  r = __builtin_fma(r, x, 1.0);
  r = __builtin_fma(r, x, 1.0);
  return ldexp(r, (int)n);
}

// ln of a positive fp64 number to about 5e-8: the exponent apart, and fp32's
// logarithm of the mantissa with the part that fp32 does not hold.
__device__ __forceinline__ double ln32(double v) {
  const double m = __builtin_amdgcn_frexp_mant(v);
  const float f = (float)m;
  const float l = hw_log2(f) + (float)(m - (double)f) * (float)kLog2e / f;
  return kLn2 * ((double)__builtin_amdgcn_frexp_exp(v) + (double)l);
}

// --- reductions over a team ------------------------------------------------------------

// Over a wave by DPP: within rows of 16 lanes, then row to row; lane 63 has
// the result, which every lane gets.
template <int CTRL, int ROWS> __device__ __forceinline__ float dpp_f(float old, float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(v), CTRL,
                                                    ROWS, 0xF, false));
}
template <int CTRL, int ROWS> __device__ __forceinline__ double dpp_d0(double v) {
  const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, ROWS, 0xF, false);
  const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, ROWS, 0xF, false);
  return __hiloint2double(hi, lo);
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), lane),
                          __builtin_amdgcn_readlane(__double2loint(v), lane));
}
__device__ __forceinline__ float wave_max(float v) {
  const float none = -__builtin_inff();
  v = fmaxf(v, dpp_f<0x111, 0xF>(none, v));
  v = fmaxf(v, dpp_f<0x112, 0xF>(none, v));
  v = fmaxf(v, dpp_f<0x114, 0xF>(none, v));
  v = fmaxf(v, dpp_f<0x118, 0xF>(none, v));
  v = fmaxf(v, dpp_f<0x142, 0xA>(none, v));
  v = fmaxf(v, dpp_f<0x143, 0xC>(none, v));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp_d0<0x111, 0xF>(v);
  v += dpp_d0<0x112, 0xF>(v);
  v += dpp_d0<0x114, 0xF>(v);
  v += dpp_d0<0x118, 0xF>(v);
  v += dpp_d0<0x142, 0xA>(v);
  v += dpp_d0<0x143, 0xC>(v);
  return lane_value(v, 63);
}
template <int NT> struct ReduceLds {
  float m[NT / kWave];
  double s[NT / kWave], w[NT / kWave];
};
// Every thread gets the result; between two uses the caller has a team_sync.
template <int NT> __device__ __forceinline__ float team_max(float v, ReduceLds<NT>& l) {
  v = wave_max(v);
  if (NT == kWave) return v;
  if (lane_id() == 0) l.m[threadIdx.x / kWave] = v;
  __syncthreads();
  v = l.m[0];
#pragma unroll
  for (int i = 1; i < NT / kWave; ++i) v = fmaxf(v, l.m[i]);
  return v;
}
// The maximum of v and whether `any` is true anywhere.
struct ListTop {
  float m;
  bool any;
};
template <int NT>
__device__ __forceinline__ ListTop team_list(float v, bool any, ReduceLds<NT>& l) {
  ListTop t{wave_max(v), __builtin_amdgcn_ballot_w64(any) != 0};
  if (NT == kWave) return t;
  if (lane_id() == 0) {
    l.m[threadIdx.x / kWave] = t.m;
    l.w[threadIdx.x / kWave] = t.any ? 1.0 : 0.0;
  }
  __syncthreads();
  t = ListTop{l.m[0], l.w[0] != 0.0};
#pragma unroll
  for (int i = 1; i < NT / kWave; ++i) {
    t.m = fmaxf(t.m, l.m[i]);
    t.any |= l.w[i] != 0.0;
  }
  return t;
}
template <int NT> __device__ __forceinline__ double team_sum(double v, ReduceLds<NT>& l) {
  v = wave_sum(v);
  if (NT == kWave) return v;
  if (lane_id() == 0) l.s[threadIdx.x / kWave] = v;
  __syncthreads();
  v = l.s[0];
#pragma unroll
  for (int i = 1; i < NT / kWave; ++i) v += l.s[i];
  return v;
}
// Sums of a whole team from those of its threads.
template <int NT, bool W>
__device__ __forceinline__ RowSums team_sums(RowSums r, float c, ReduceLds<NT>& l) {
  const float m = team_max<NT>(r.m, l);
  sums_move<W>(r, c, m);
  r.s = wave_sum(r.s);
  if (W) r.w = wave_sum(r.w);
  if (NT == kWave) return r;
  if (lane_id() == 0) {
    l.s[threadIdx.x / kWave] = r.s;
    if (W) l.w[threadIdx.x / kWave] = r.w;
  }
  __syncthreads();
  r.s = l.s[0];
  if (W) r.w = l.w[0];
#pragma unroll
  for (int i = 1; i < NT / kWave; ++i) {
    r.s += l.s[i];
    if (W) r.w += l.w[i];
  }
  return r;
}
// A part of a row, whichever kind it is.  The last barrier is before the last
// reads of l.
template <typename E, int NT, bool W, bool LISTED, bool ONCE, int HG, bool ALL>
__device__ __forceinline__ RowSums part_sums(const Part<E>& part, float c, const uint32_t* listed,
                                             float* gmax, RowStart<E, HG>& start, float& mine,
                                             ReduceLds<NT>& l) {
  RowSums r = row_sums<E, NT, W, LISTED, ONCE, HG, ALL>(part, c, listed, gmax, start);
  mine = r.m;
  r = team_sums<NT, W>(r, c, l);
  if (far_row(r.m, c)) {
    r = row_sums_far<E, NT, W, LISTED>(part, c, r.m, listed);
    team_sync<NT>();
    r.s = team_sum<NT>(r.s, l);
    if (W) {
      team_sync<NT>();
      r.w = team_sum<NT>(r.w, l);
    }
  }
  return r;
}
// Joins sums of parts, each against the reference of its own maximum, far or
// not, in `r`.
template <bool W> __device__ __forceinline__ void sums_join(RowSums& r, RowSums o, float c) {
  const float m = fmaxf(r.m, o.m);
  auto to_m = [&](RowSums& a) {
    if (a.m != m && a.m != -__builtin_inff()) {   // below every entry: sums of zero, or NaN
      const float d = (float)(reference64(a.m, c) - reference64(m, c));
      const double f = (double)hw_exp2(d);
      if (W) a.w = f == 0.0 ? f * a.w : f * (a.w + (double)d * a.s);
      a.s *= f;
    }
    a.m = m;
  };
  to_m(r);
  to_m(o);
  r.s += o.s;
  if (W) r.w += o.w;
}
// Over a team, every thread with the join of some parts.
template <int NT, bool W>
__device__ __forceinline__ RowSums team_join(RowSums r, float c, ReduceLds<NT>& l) {
  RowSums all{team_max<NT>(r.m, l), 0.0, 0.0};
  sums_join<W>(r, all, c);
  team_sync<NT>();
  r.s = team_sum<NT>(r.s, l);
  if (W) {
    team_sync<NT>();
    r.w = team_sum<NT>(r.w, l);
  }
  return r;
}

// --- the largest entries ---------------------------------------------------------------------

// Order of the entries as integers: by value (-0 as +0, a NaN as -inf), ties
// to the lower index.
__device__ __forceinline__ uint32_t value_order(float v) {
  v = v != v ? -__builtin_inff() : v + 0.f;
  const uint32_t b = __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint64_t entry_key(uint32_t order, uint32_t index) {
  return ((uint64_t)order << 32) | (uint32_t)~index;
}
__device__ __forceinline__ uint32_t key_index(uint64_t key) { return ~(uint32_t)key; }
__device__ __forceinline__ float key_value(uint64_t key) {
  return order_value((uint32_t)(key >> 32));
}

constexpr int kTopMax = 128;        // entries asked for
constexpr int kTopWave = 48;        // by a team of one wave, of any row

template <int NT> struct alignas(16) TopLds {
  static constexpr int kOrders = NT < 256 ? NT : 256;
  // (Where fewer threads than k have a vector, all their entries are candidates:
  // 47 vectors and 14 entries beside them for a wave, 127 for a block of 256.)
  static constexpr int kCandidates = NT < 256 ? 512 : NT == 256 ? 1280 : 2048;
  static constexpr int kGroups = NT < 256 ? 64 : 512;
  uint32_t order[kOrders];
  uint32_t group[kGroups];
  uint32_t floor, count, above, groups;
  uint64_t cand[kCandidates];
  uint64_t best[kTopMax];
};

// The k-th largest of the threads' orders (0: the thread has no entry), a
// bound that k entries reach, and in a row whose large entries lie anywhere
// only a few more do: of n maxima, n ln(n / (n - k)) on average, 24 for the
// 20th of 64, 89 for the 64th of 128.  Maxima of lanes next to each other are
// joined where fewer than all are enough: the comparisons grow with the square
// of their number.
// `have`: threads 0 .. have - 1 are those with an entry.
template <int NT>
__device__ __forceinline__ uint32_t top_floor(uint32_t order, uint32_t have, int k, TopLds<NT>& l) {
  const uint32_t tid = team_tid<NT>();
  if (tid == 0) {
    // (More entries than a wave has maxima: no bound.)
    l.floor = NT == kWave && k > kWave ? 0u : 0xFFFFFFFFu;
    l.count = l.above = l.groups = 0;
  }
  // One order for each G lanes, which share its comparisons with the others.
  auto bound_of = [&](auto groups) {
    constexpr int NO = decltype(groups)::value, G = NT / NO, per = NO / G;
    uint32_t o = order;
#pragma unroll
    for (int d = 1; d < G; d <<= 1) o = max(o, (uint32_t)__shfl_xor((int)o, d));
    if (tid % G == 0) l.order[tid / G] = o;
    team_sync<NT>();
    int above = 0;
    const uint32_t* from = &l.order[(tid % G) * per];
#pragma unroll
    for (int i = 0; i < per; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(from + i);
      above += (v.x > o) + (v.y > o) + (v.z > o) + (v.w > o);
    }
#pragma unroll
    for (int d = 1; d < G; d <<= 1) above += __shfl_xor(above, d);
    if (tid % G == 0 && above < k) atomicMin(&l.floor, o);
    team_sync<NT>();
  };
  // Enough: a third more maxima than k.
  const uint32_t want = 4u * (uint32_t)k * NT;
  if (NT == kWave || have * 64 * 3 >= want) bound_of(std::integral_constant<int, 64>());
  else if (have * 128 * 3 >= want) bound_of(std::integral_constant<int, NT < 256 ? NT : 128>());
  else bound_of(std::integral_constant<int, NT < 256 ? NT : 256>());
  return l.floor;
}

// Puts a key into the candidates' list (count may pass its length; the
// comparison of count with it comes behind a team_sync).
template <int NT> __device__ __forceinline__ void top_push(uint64_t key, TopLds<NT>& l) {
  const uint32_t at = atomicAdd(&l.count, 1u);
  if (at < TopLds<NT>::kCandidates) l.cand[at] = key;
}

// The k largest of l.cand[0, count) in falling order, in l.best: the rank of a
// candidate is the number of larger ones.  A long list is cut by the bound
// among its own maxima first.
template <int NT> __device__ __forceinline__ void top_rank(uint32_t count, int k, TopLds<NT>& l) {
  const uint32_t tid = team_tid<NT>();
  if (count > NT || count > 256) {
    constexpr int per = TopLds<NT>::kCandidates / NT;
    uint64_t mine[per], largest = 0;
#pragma unroll
    for (int i = 0; i < per; ++i) {
      mine[i] = tid + i * NT < count ? l.cand[tid + i * NT] : 0;
      largest = max(largest, mine[i]);
    }
    team_sync<NT>();
    const uint32_t floor = top_floor<NT>((uint32_t)(largest >> 32), min(count, (uint32_t)NT), k, l);
#pragma unroll
    for (int i = 0; i < per; ++i)
      if (mine[i] && (uint32_t)(mine[i] >> 32) >= floor) l.cand[atomicAdd(&l.count, 1u)] = mine[i];
    team_sync<NT>();
    count = l.count;
  }
  const uint32_t even = (count + 3) & ~3u;
  if (tid < even - count) l.cand[count + tid] = 0;
  team_sync<NT>();
  for (uint32_t i = tid; i < count; i += NT) {
    const uint64_t key = l.cand[i];
    int rank = 0;
    for (uint32_t j = 0; j < even; j += 4) {
      const ulonglong2 p = *reinterpret_cast<const ulonglong2*>(&l.cand[j]);
      const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(&l.cand[j + 2]);
      rank += (p.x > key) + (p.y > key) + (q.x > key) + (q.y > key);
    }
    if (rank < k) l.best[rank] = key;
  }
  team_sync<NT>();
}

// Calls f(key) for each of the calling thread's entries of a part of a row
// whose group's maximum (gmax of row_sums) has an order of at_least or more.
template <typename E, int NT, typename F>
__device__ __forceinline__ void each_key(const Part<E>& part, const float* gmax, uint32_t at_least,
                                         F f) {
  constexpr int n = kRowVec<E>, U = kRowUnroll<E>;
  const uint32_t nvec = part.nvec, tid = team_tid<NT>(), first = part.lo + part.head;
  for (uint32_t base = 0; base < nvec; base += U * NT) {
    if (value_order(gmax[base / U + tid]) < at_least) continue;
    const Group<E> g = group_load<E, NT>(part.vectors(), base, nvec);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t v = base + u * NT + tid;
      const auto x = row_wide<E>(g.v[u]);
      if (v < nvec)
#pragma unroll
        for (int i = 0; i < n; ++i) f(entry_key(value_order(x[i]), first + v * n + i));
    }
  }
  const uint32_t rest = part.rest(tid);
  if (rest < part.len) f(entry_key(value_order((float)part.z[rest]), part.lo + rest));
}

// The k largest entries' keys of a part of a row (of k entries or more) in
// falling order, in l.best, from the groups' maxima that row_sums left and
// the calling thread's own maximum (order; 0: it has no entry).
//
// The groups that reach the bound of top_floor are listed and their vectors
// read once more, a vector a thread, so that their loads are all under way
// together; the candidates' ranks come from comparing each with each.
//
// Lists overflow where values repeat at the bound, or where the large entries
// share few threads.  Then, with `above` entries beyond the bound: if they fit,
// the ties are taken from the lower ids up (a constant row needs one look);
// else the k-th key itself is found bit by bit, a pass over the part for each.
template <typename E, int NT>
__device__ __forceinline__ void top_entries(const Part<E>& part, const float* gmax, uint32_t order,
                                            int k, TopLds<NT>& l) {
  constexpr int n = kRowVec<E>, U = kRowUnroll<E>;
  constexpr uint32_t most = TopLds<NT>::kCandidates;
  const uint32_t tid = team_tid<NT>(), nvec = part.nvec, lo = part.lo;
  const uint32_t have = min((uint32_t)NT, max(nvec, part.rests()));
  const uint32_t floor = top_floor<NT>(order, have, k, l);
  for (uint32_t base = 0; base < nvec; base += U * NT)
    if (base + tid < nvec && value_order(gmax[base / U + tid]) >= floor) {
      const uint32_t at = atomicAdd(&l.groups, 1u);
      if (at < TopLds<NT>::kGroups) l.group[at] = base / U + tid;
    }
  const uint32_t rest = part.rest(tid);
  if (rest < part.len) {
    const uint32_t o = value_order((float)part.z[rest]);
    if (o >= floor) top_push<NT>(entry_key(o, lo + rest), l);
  }
  team_sync<NT>();
  const uint32_t groups = l.groups;
  if (groups <= TopLds<NT>::kGroups) {
    for (uint32_t i = tid; i < groups * U; i += NT) {
      const uint32_t at = l.group[i / U];
      const uint32_t v = (at / NT) * (U * NT) + (i % U) * NT + at % NT;
      if (v >= nvec) continue;
      const auto x = row_wide<E>(row_load<E>(part.vectors() + (size_t)v * n));
      int mine = 0;
#pragma unroll
      for (int j = 0; j < n; ++j) mine += value_order(x[j]) >= floor;
      if (mine == 0) continue;
      uint32_t put = atomicAdd(&l.count, (uint32_t)mine);
#pragma unroll
      for (int j = 0; j < n; ++j) {
        const uint32_t o = value_order(x[j]);
        if (o >= floor && put < most) l.cand[put++] = entry_key(o, lo + part.head + v * n + j);
      }
    }
    team_sync<NT>();
    if (l.count <= most) {
      top_rank<NT>(l.count, k, l);
      return;
    }
  }
  // Entries of the team for which `test` is true, counted in a word of LDS.
  auto count_if = [&](uint32_t& word, uint32_t at_least, auto test) {
    uint32_t mine = 0;
    each_key<E, NT>(part, gmax, at_least, [&](uint64_t key) { mine += test(key); });
    team_sync<NT>();
    if (tid == 0) word = 0;
    team_sync<NT>();
    if (mine) atomicAdd(&word, mine);
    team_sync<NT>();
    return word;
  };
  const uint64_t ties = ((uint64_t)floor << 32) | 0xFFFFFFFFu;   // keys above it: entries beyond
  const uint32_t above = count_if(l.above, floor, [&](uint64_t key) { return key > ties; });
  uint64_t bound = ties + 1;                 // keys from it up are candidates
  if (above + NT > most) {
    // The largest key that k keys reach, from its highest bit down.
    bound = 0;
    for (int bit = 63; bit >= 0; --bit) {
      const uint64_t tried = bound | (1ull << bit);
      const uint32_t reach = count_if(l.above, (uint32_t)(tried >> 32),
                                      [&](uint64_t key) { return key >= tried; });
      if (reach >= (uint32_t)k) bound = tried;
    }
  }
  team_sync<NT>();
  if (tid == 0) l.count = 0;
  team_sync<NT>();
  each_key<E, NT>(part, gmax, (uint32_t)(bound >> 32), [&](uint64_t key) {
    if (key >= bound) top_push<NT>(key, l);
  });
  team_sync<NT>();
  for (uint32_t base = 0; base < part.len && l.count < (uint32_t)k; base += NT) {
    team_sync<NT>();                         // every thread has seen the count
    if (base + tid < part.len && value_order((float)part.z[base + tid]) == floor)
      top_push<NT>(entry_key(floor, lo + base + tid), l);
    team_sync<NT>();
  }
  team_sync<NT>();
  top_rank<NT>(min(l.count, most), k, l);
}

// The same for n keys in memory (0: none), k of them or more not zero.
template <int NT>
__device__ __forceinline__ void top_of_keys(const uint64_t* keys, uint32_t n, int k,
                                            TopLds<NT>& l) {
  const uint32_t tid = team_tid<NT>();
  uint64_t largest = 0;
  for (uint32_t i = tid; i < n; i += NT) largest = max(largest, keys[i]);
  const uint32_t floor = top_floor<NT>((uint32_t)(largest >> 32), min(n, (uint32_t)NT), k, l);
  for (uint32_t i = tid; i < n; i += NT)
    if (keys[i] && (uint32_t)(keys[i] >> 32) >= floor) top_push<NT>(keys[i], l);
  team_sync<NT>();
  if (l.count <= TopLds<NT>::kCandidates) {
    top_rank<NT>(l.count, k, l);
    return;
  }
  uint64_t bound = 0;
  for (int bit = 63; bit >= 0; --bit) {
    const uint64_t tried = bound | (1ull << bit);
    uint32_t mine = 0;
    for (uint32_t i = tid; i < n; i += NT) mine += keys[i] >= tried;
    team_sync<NT>();
    if (tid == 0) l.count = 0;
    team_sync<NT>();
    if (mine) atomicAdd(&l.count, mine);
    team_sync<NT>();
    if (l.count >= (uint32_t)k) bound = tried;
  }
  team_sync<NT>();
  if (tid == 0) l.count = 0;
  team_sync<NT>();
  for (uint32_t i = tid; i < n; i += NT)
    if (keys[i] && keys[i] >= bound) top_push<NT>(keys[i], l);
  team_sync<NT>();
  top_rank<NT>(l.count, k, l);
}

// Bytes of gmax for a part of `len` entries.
template <typename E, int NT> __host__ __device__ inline size_t gmax_bytes(uint32_t len) {
  const uint32_t step = kGroup<E> * NT;
  return (size_t)((len + step - 1) / step) * NT * 4;
}

// --- host side -----------------------------------------------------------------------------

// Temperatures the kernels take: the scaled exponents stay in fp32's range.
constexpr double kTemperatureMin = 1e-6, kTemperatureMax = 1e6;
inline bool temperature_ok(double t) { return t >= kTemperatureMin && t <= kTemperatureMax; }
inline float make_scale(double temperature) { return (float)(kLog2e / temperature); }

// Who works on a row of V entries: a team of `nt` threads, or, where a row is
// longer than kPartMax (the bitmap of a part is 16 KiB of LDS; its groups'
// maxima, for the top entries, are 16 KiB of 16-bit logits and 32 of fp32),
// `parts` blocks with `len` entries each, joined by a second kernel.
// `wave`: longest row that a wave takes by itself (4096 rows of 4096: 10 us by
// waves, 17 by blocks of 256).  Blocks of 512 where a CU (of an MI355X's 256)
// has one row at most: loss and gradient of 200 rows of 65537 take 19.4 us by 512 and 22.0
// by 256, their values 10 by both; 256 rows of 131072 38.1 and 39.9, values
// 16.4 and 14.9.  With more rows, blocks of 256: 300 rows of 65537 take 29.6 us
// against 32.2, 511 rows of 131072 60 against 68, values 25 against 29, 700 of
// 65537 41 against 53.  (At 65537 entries blocks of either size read a part of a
// row twice; whether 512 threads that hold all of it would win is not measured.)
// One row of 131072 is one block's work too: 13 us, and 13.6 in parts with their
// join; a few rows of that length were not compared.
constexpr uint32_t kPartMax = SDTW_ROWS_WHOLE;
struct Split {
  uint32_t parts, len;
  int nt;
};
inline Split split_rows(int64_t rows, int64_t V, int64_t wave) {
  if (V > kPartMax) {
    int64_t parts = (V + (1 << 15) - 1) >> 15;             // few rows: more blocks
    if (parts > (512 + rows - 1) / rows) parts = (512 + rows - 1) / rows;
    if (parts < (V + kPartMax - 1) / kPartMax) parts = (V + kPartMax - 1) / kPartMax;
    const int64_t len = ((V + parts - 1) / parts + 63) / 64 * 64;
    return Split{(uint32_t)((V + len - 1) / len), (uint32_t)len, 512};
  }
  const int nt = V <= wave && rows >= 1024 ? 64 : rows > 256 || V <= 16384 ? 256 : 512;
  return Split{1, (uint32_t)V, nt};
}

// Entries of a row one team of a gradient kernel writes: one group.
template <typename E> inline void grad_chunks(int64_t V, int nt, uint32_t* chunks, uint32_t* len) {
  const int64_t most = (int64_t)nt * kGroup<E>;
  *len = (uint32_t)(V < most ? V : most);
  *chunks = (uint32_t)((V + *len - 1) / *len);
}

inline bool dtype_ok(int dtype) { return dtype >= SDTW_DTYPE_F32 && dtype <= SDTW_DTYPE_F16; }
// Sizes the kernels' 32-bit row and entry numbers hold.
inline bool rows_ok(int64_t B, int64_t N, int64_t V) {
  const int64_t most = (int64_t(1) << 31) - 1;
  return B >= 1 && N >= 1 && V >= 1 && B <= most && N <= most && V <= most && B * N <= most;
}
inline RowsIn rows_in(const void* z, int64_t B, int64_t N, int64_t V, int64_t ld_b, int64_t ld_n) {
  return RowsIn{z, ld_b, ld_n, (uint32_t)(B * N), (uint32_t)N, (uint32_t)V};
}

// Whether logits (and a gradient of their size) are read and written past the
// caches: they and the gradient do not fit in the 256 MiB last-level cache, so
// that nothing of them is there at their next use.  Reading 1 GiB takes 170 us
// past the caches and 220 us through them; 65 MB that the cache holds take 22
// us through it and 30 us past it.
inline bool read_once(const RowsIn& a, size_t size) {
  return (size_t)a.rows * a.V * size > (size_t(128) << 20);
}

// One launch of `f(first item, blocks)` for every 2^22 blocks of `teams` items
// each: a grid has at most 2^32 threads.  (A loop over items inside a kernel
// costs registers: it keeps the constants of the fp64 functions in them.)
template <typename F> inline hipError_t launch_items(uint64_t items, int teams, F f) {
  const uint64_t most = (uint64_t)(1u << 22) * teams;
  for (uint64_t first = 0; first < items; first += most) {
    const uint64_t n = items - first < most ? items - first : most;
    f(first, (uint32_t)((n + teams - 1) / teams));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace sdtw
