// Distillation of a row of logits from a teacher's list of likely entries
// (sdtw_distill_* of include/sdtw.h): loss, gradient, or both at once.
//
// With p = softmax(z / T) of the row and q the teacher's probabilities of the
// list's entries,
//   without the tail:  q = softmax of the list / T,
//     L = sum_k q_k (log q_k - log p_k),        T dL/dz_j = p_j - q_j
//     (q_j = 0 off the list);
//   with the tail:     q_k = e^(list value), q_r = 1 - sum_k q_k, and p_r the
//     row's probability off the list,
//     L = sum_k q_k (log q_k - log p_k) + q_r (log q_r - log p_r),
//     T dL/dz_j = p_j - q_j on the list,  p_j (1 - q_r / p_r) off it.
// An id that stands twice in a list counts once in p and adds in q.  p_r is
// summed over the entries off the list themselves (a difference from one
// would lose it where the student is sure of the list): a bitmap of the list
// in LDS costs one byte's read for each vector of logits.  Their exponents'
// reference is their own maximum, m_r, so that neither p_r nor its logarithm is
// ever too small for the numbers they are held in: with S_r their sum,
//   p_r = S_r 2^(m_r - m) / S,  T dL/dz_j = 2^(t_j - m_r) (p_r - q_r) / S_r.
// The loss is a
// small difference of logarithms once the student is near the teacher, so
// the sums and the list's few values are fp64.
#include "sdtw.h"
#include "sdtw_kernels.h"
#include "sdtw_rows.h"

namespace sdtw {
namespace {

constexpr int kListMax = 256;   // one entry of the list per thread
constexpr int kListWave = 64;   // of a team of one wave

// What the gradient needs of a row.
struct alignas(16) DistillStats {
  float ref;      // reference of the exponents
  float inv_s;    // 1 / sum of the row (0: no entry above -inf)
  float off;      // factor of 2^t off the list (NaN: a bad id)
  float tmax;     // q = e^((t - tmax) * tscale) * qscale
  float tscale, qscale;
  float far;      // exponents as (z - ref) c: 1 against ref, 2 against off_ref
  float off_ref;  // reference of the exponents off the list
};

struct DistillArgs {
  RowsIn in;
  uint64_t first;          // item of the launch's first team
  IdsIn ids;               // [rows, K]
  IdsIn list;              // the teacher's values; bytes: their dtype
  int64_t ignore;
  float c;
  double inv_t;
  int K;
  Split split;
  RowSums* part;           // [rows, parts] (parts > 1)
  float* loss;             // [rows]
  DistillStats* stats;     // [rows] or null
  const float* weight;     // upstream gradient of each row, w_step apart; null: 1
  int64_t w_step;
  uint32_t chunks, len;    // gradient kernel: teams of a row, entries of each
  void* grad;              // [rows, V]
};

__device__ __forceinline__ float list_load(const DistillArgs& a, uint32_t row, uint32_t k) {
  const uint32_t n = a.in.n, q = n >= a.in.rows ? 0 : row / n;
  const int64_t i = (int64_t)q * a.list.ld0 + (int64_t)(row - q * n) * a.list.ld1 + k;
  if (a.list.bytes == SDTW_DTYPE_F32) return static_cast<const float*>(a.list.p)[i];
  if (a.list.bytes == SDTW_DTYPE_BF16) return (float)static_cast<const __bf16*>(a.list.p)[i];
  return (float)static_cast<const _Float16*>(a.list.p)[i];
}

// The list of a row in LDS: ids (-1: none), and the teacher's probabilities.
template <int NT> struct alignas(16) DistillLds {
  static constexpr int kList = NT < 256 ? kListWave : kListMax;
  int ids[kList];
  float q[kList];
  int twice;       // whether an id stands twice (TAIL)
};

// The calling thread's entry of the list, loaded early.
struct ListEntry {
  int id;          // -1: none (padding), -2: outside the vocabulary
  float t, z;      // the teacher's value; the row's logit there
};
__device__ __forceinline__ int list_id(const DistillArgs& a, uint32_t row, int tid) {
  if (tid >= a.K) return -1;
  const int64_t id = id_load(a.ids, a.in.rows, a.in.n, row, tid);
  return id == a.ignore ? -1 : id >= 0 && id < (int64_t)a.in.V ? (int)id : -2;
}
template <typename E>
__device__ __forceinline__ ListEntry list_entry(const DistillArgs& a, uint32_t row, int tid,
                                                int id) {
  ListEntry e{id, -__builtin_inff(), 0.f};
  if (id != -1) e.t = list_load(a, row, tid);
  if (id >= 0) e.z = (float)row_ptr<E>(a.in, row)[id];
  return e;
}

// Loss and statistics of a row by a team, thread k with the list's k-th entry
// (`first`: the first, or only, entry of its id), from the row's maximum and
// its sum (those of the entries off the list if TAIL).  Returns the statistics
// and the thread's q.
template <typename E, bool TAIL, int NT>
__device__ __forceinline__ DistillStats distill_finish(const DistillArgs& a, uint32_t row,
                                                       RowSums r, const ListEntry& e, bool first,
                                                       float& q32, ReduceLds<NT>& l) {
  const int tid = team_tid<NT>();
  // fmax passes over a NaN of the teacher, or of the listed logits; the sums
  // below meet it again.
  float tmax = 0.f, m = r.m;
  bool listed = false;
  if (TAIL) {
    const ListTop t = team_list<NT>(e.id >= 0 ? e.z : -__builtin_inff(), e.id != -1, l);
    m = fmaxf(m, t.m);
    listed = t.any;
  } else {
    tmax = team_max<NT>(e.t, l);
    if (tmax == -__builtin_inff()) tmax = 0.f;
  }
  const Exponent x = row_exponent(m, a.c), y = TAIL ? row_exponent(r.m, a.c) : x;
  const double tscale = TAIL ? 1.0 : a.inv_t;
  const double u = ((double)e.t - (double)tmax) * tscale;
  double q = e.id != -1 ? exp(u) : 0.0;
  team_sync<NT>();
  const double qsum = team_sum<NT>(q, l);
  // Nothing listed, or (without the tail) every entry of zero probability: no
  // teacher, and neither loss nor gradient whatever the logits hold.
  const bool teacher = TAIL ? listed : qsum != 0.0;
  const double t2 = exponent64(x, e.z);
  double sum = r.s, share = r.s, down = 0.0;
  if (TAIL) {
    // The share of the entries off the list (none of them above -inf: zero, or
    // NaN), and the list's own, every id once.
    down = reference64(r.m, a.c) - reference64(m, a.c);
    if (r.m != -__builtin_inff()) share *= exp2_wide(down);
    team_sync<NT>();
    sum = share + team_sum<NT>(first && e.id >= 0 ? (double)hw_exp2((float)t2) : 0.0, l);
  }
  const bool none = sum == 0.0 && m == -__builtin_inff();
  double rest = TAIL && teacher ? 1.0 - qsum : 0.0;
  if (rest < 0.0) rest = 0.0;
  const double inv = none ? 0.0 : 1.0 / sum;
  const double left = TAIL ? share * inv : 0.0;
  // One evaluation of the logarithm, on four lanes.
  const int lane = lane_id();
  const double lns = log(lane == 0 ? sum : lane == 1 ? qsum : lane == 2 ? rest : r.s);
  const double ln_s = none ? 0.0 : lane_value(lns, 0);
  const double logp = none ? -kInf : kLn2 * t2 - ln_s;
  double logq = u, qscale = 1.0;
  if (!TAIL) {
    qscale = teacher ? 1.0 / qsum : 0.0;
    logq = u - (teacher ? lane_value(lns, 1) : 0.0);
    q *= qscale;
  }
  q32 = (float)q;
  double part = q == 0.0 ? 0.0 : q * (logq - logp);
  if (e.id == -2) part = __builtin_nan("");
  team_sync<NT>();
  double loss = team_sum<NT>(part, l);
  double off = teacher ? inv : 0.0;
  if (TAIL && teacher) {
    if (left < 0x1p-126 && !none) {
      // Next to nothing off the list for the rest to fall on: what roundings can
      // make of a list that is complete is no rest.  Its values are off by half
      // a step of their type each, and all of them together by what fp32 leaves
      // of the log-sum-exp that was taken from them: half a step of it, up to
      // 2^-19 for logits up to 64, and as much again for its sum.
      const double half = a.list.bytes == SDTW_DTYPE_F32    ? 0x1p-24
                          : a.list.bytes == SDTW_DTYPE_BF16 ? 0x1p-8 : 0x1p-11;
      team_sync<NT>();
      if (rest <= 0x1p-18 + half * (1.0 + team_sum<NT>(q == 0.0 ? 0.0 : q * fabs(logq), l)))
        rest = 0.0;
    }
    if (rest != 0.0)
      loss += rest * (lane_value(lns, 2) - (lane_value(lns, 3) + kLn2 * down - ln_s));
    // (No entry off the list: nothing to scale.)
    off = r.s == 0.0 ? 0.0 : (left - rest) / r.s;
  }
  if (__builtin_isnan(loss)) off = __builtin_nan("");
  if (none) qscale = 0.0;
  const DistillStats st{x.ref, (float)inv, none ? 0.f : (float)off, tmax, (float)tscale,
                        (float)qscale, (x.far ? 1.f : 0.f) + (y.far ? 2.f : 0.f), y.ref};
  if (tid == 0) {
    a.loss[row] = (float)loss;
    if (a.stats) a.stats[row] = st;
  }
  return st;
}

// Writes the gradient of a part of a row, first as of entries off the list
// (whose reference a listed entry may exceed by any amount: what is written for
// it is whatever comes of that), then the list's own.  `id` is the calling
// thread's entry of the
// list (-1: none), whose ids and probabilities are in l behind a team_sync.
// The first HG groups (ALL: there are no more) are in `held` already.
template <typename E, int NT, bool ONCE, int HG, bool ALL>
__device__ __forceinline__ void distill_grad(const DistillArgs& a, uint32_t row,
                                             const Part<E>& part, const DistillStats& st, int id,
                                             const DistillLds<NT>& l, const Group<E>* held) {
  constexpr int n = kRowVec<E>, U = kRowUnroll<E>, step = U * NT;
  const uint32_t tid = team_tid<NT>(), nvec = part.nvec;
  const E* z = part.z;
  E* out = static_cast<E*>(a.grad) + (size_t)row * a.in.V + part.lo;
  const float w = (a.weight ? a.weight[(size_t)row * a.w_step] : 1.f) * (float)a.inv_t;
  const float on = w * st.inv_s, A = st.off == 0.f ? 0.f : w * st.off;
  const Exponent on_list{a.c, st.ref, st.far == 1.f || st.far == 3.f};
  const Exponent ex{a.c, st.off_ref, st.far >= 2.f};
  auto write = [&](auto value) {
    auto group = [&](const Group<E>& g, uint32_t base) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t v = base + u * NT + tid;
        auto x = row_wide<E>(g.v[u]);
#pragma unroll
        for (int i = 0; i < n; ++i) x[i] = value(x[i]);
        if (v < nvec) row_store<E, ONCE>(out + part.head + (size_t)v * n, x);
      }
    };
    Group<E> ga, gb;
    if (!ALL && HG * step < nvec) {
      ga = group_load<E, NT, ONCE>(part.vectors(), HG * step, nvec);
      gb = group_load<E, NT, ONCE>(part.vectors(), (HG + 1) * step, nvec);
    }
#pragma unroll
    for (int h = 0; h < HG; ++h)
      if (h * step < nvec) group(held[h], h * step);
    if (!ALL) each_group<E, NT, ONCE>(part.vectors(), HG * step, nvec, ga, gb, group);
    const uint32_t rest = part.rest(tid);
    if (rest < part.len) out[rest] = (E)value((float)z[rest]);
  };
  // A row of no weight, or whose entries off the list have no gradient.
  if (w == 0.f || A == 0.f) write([](float) { return 0.f; });
  else if (ex.far) write([&](float x) { return hw_exp2(exponent<true>(ex, x)) * A; });
  else write([&](float x) { return hw_exp2(exponent<false>(ex, x)) * A; });
  team_sync<NT>();
  const int lo = (int)part.lo;
  if (w != 0.f && st.inv_s != 0.f && st.qscale != 0.f && !__builtin_isnan(A) && id >= lo &&
      id < lo + (int)part.len) {
    float q = 0.f;                      // every entry of the same id writes the same sum
    for (int j = 0; j < a.K; ++j) q += l.ids[j] == id ? l.q[j] : 0.f;
    const float x = (float)z[id - lo];
    const float t = on_list.far ? exponent<true>(on_list, x) : exponent<false>(on_list, x);
    out[id - lo] = (E)(hw_exp2(t) * on - w * q);
  }
}

// One part of a row per team; a whole row (parts == 1) is finished here, with
// GRAD its gradient too: from its first HG groups, which stayed in registers,
// and a second look at the others (ALL: there are none).
//
// Values: bound by memory, and by the row's own chain (list, sums, logarithms)
// where rows are short.  4096 rows of 131072 (bf16), K = 64: 163 us, 6.6 TB/s;
// with the tail 183, since its list has to be in the bitmap before the first
// sum.  2048 rows of 50016: 41 us, with the tail 46.  With the gradient: 455 us
// for the 4096, against 163 + 350 in two launches; 1.8 GiB read and 1 written,
// bound by the last-level cache and memory together.  513 rows of 65537
// (fp16), K = 128: 40 us.
template <typename E, bool TAIL, bool GRAD, int HG, bool ALL, int NT, bool ONCE>
__global__ __launch_bounds__(kTeamBlock<NT>) void
k_distill_rows(DistillArgs a) {
  __shared__ ReduceLds<NT> red;          // (a wave reduces in registers)
  __shared__ DistillLds<NT> lists[GRAD || TAIL ? kTeams<NT> : 1];
  extern __shared__ uint32_t bits[];     // TAIL: a bit for each entry of the part
  const uint32_t words = bitmap_words<E>(a.split.len);
  uint32_t* listed = bits + team_id<NT>() * words;
  DistillLds<NT>& l = lists[GRAD || TAIL ? team_id<NT>() : 0];
  const uint32_t tid = team_tid<NT>();
  const uint64_t items = (uint64_t)a.in.rows * a.split.parts;
  const uint64_t item = a.first + (uint64_t)blockIdx.x * kTeams<NT> + team_id<NT>();
  if (item >= items) return;
  const uint32_t row = a.split.parts == 1 ? (uint32_t)item : (uint32_t)(item / a.split.parts);
  const uint32_t lo = (uint32_t)(item - (uint64_t)row * a.split.parts) * a.split.len;
  const uint32_t hi = min(a.in.V, lo + a.split.len);
  const E* z = row_ptr<E>(a.in, row);
  const Part<E> p = make_part<E>(z, lo, hi, z + lo);
  // The list's ids are asked for first, the row's first groups behind them;
  // the list is then at hand while those are on their way.
  constexpr bool PAST = ONCE && (ALL || !GRAD);     // a row that is not read again
  const int id = list_id(a, row, tid);
  auto start = row_start<E, NT, PAST, HG, ALL>(p);
  __builtin_amdgcn_sched_barrier(0);
  bool first = true;
  if (TAIL) {
    for (uint32_t i = tid; i < words; i += NT) listed[i] = 0;
    if (tid < DistillLds<NT>::kList) l.ids[tid] = id;
    if (tid == 0) l.twice = 0;
    team_sync<NT>();
    stress_delay(64);
    if (id >= (int)lo && id < (int)hi) {
      const uint32_t at = p.bit(id - lo), bit = 1u << (at & 31);
      if (atomicOr(&listed[at >> 5], bit) & bit) l.twice = 1;
    }
    team_sync<NT>();
    // Of equal ids the first one counts, not the one whose wave came first: the
    // order of the list's sum goes by the list alone.
    if (l.twice && id >= 0)
      for (int j = 0; j < (int)tid; ++j) first &= l.ids[j] != id;
  }
  const ListEntry e = list_entry<E>(a, row, tid, id);
  float mine;
  const RowSums r =
      part_sums<E, NT, false, TAIL, PAST, HG, ALL>(p, a.c, listed, nullptr, start, mine, red);
  if (a.split.parts > 1) {
    if (tid == 0) a.part[item] = r;
  } else {
    float q;
    team_sync<NT>();
    const DistillStats st = distill_finish<E, TAIL, NT>(a, row, r, e, first, q, red);
    if (GRAD) {
      if (tid < DistillLds<NT>::kList) {
        l.ids[tid] = e.id;
        l.q[tid] = q;
      }
      team_sync<NT>();
      distill_grad<E, NT, ONCE, HG, ALL>(a, row, p, st, e.id, l, start.held);
    }
  }
}

// Joins the parts of a row and takes its loss: a block a row, bound by latency.
template <typename E, bool TAIL>
__global__ __launch_bounds__(256) void k_distill_join(DistillArgs a) {
  constexpr int NT = 256;
  __shared__ ReduceLds<NT> red;
  __shared__ int ids[kListMax];
  const uint32_t row = (uint32_t)a.first + blockIdx.x;
  RowSums mine{-__builtin_inff(), 0.0, 0.0};
  for (uint32_t i = threadIdx.x; i < a.split.parts; i += NT)
    sums_join<false>(mine, a.part[(size_t)row * a.split.parts + i], a.c);
  const ListEntry e = list_entry<E>(a, row, threadIdx.x, list_id(a, row, threadIdx.x));
  ids[threadIdx.x] = e.id;
  const RowSums r = team_join<NT, false>(mine, a.c, red);
  bool first = true;
  if (TAIL && e.id >= 0)
    for (int j = 0; j < (int)threadIdx.x; ++j) first &= ids[j] != e.id;
  float q;
  __syncthreads();
  distill_finish<E, TAIL, NT>(a, row, r, e, first, q, red);
}

// The gradient from the statistics, a team for each group of a row.  Bound by
// memory, one read and one write: 4096 rows of 131072 (bf16) take 350 us, 6.1
// TB/s; 1000 rows of 50021 (fp32) 73 us, 5.5 TB/s.
template <typename E, int NT, bool ONCE> __global__ __launch_bounds__(256) void
k_distill_grad(DistillArgs a) {
  __shared__ DistillLds<NT> lists[kTeams<NT>];
  DistillLds<NT>& l = lists[team_id<NT>()];
  const uint32_t tid = team_tid<NT>();
  const uint64_t items = (uint64_t)a.in.rows * a.chunks;
  const uint64_t item = a.first + (uint64_t)blockIdx.x * kTeams<NT> + team_id<NT>();
  if (item >= items) return;
  const uint32_t row = a.chunks == 1 ? (uint32_t)item : (uint32_t)(item / a.chunks);
  const uint32_t lo = (uint32_t)(item - (uint64_t)row * a.chunks) * a.len;
  const uint32_t hi = min(a.in.V, lo + a.len);
  const Part<E> p = make_part<E>(row_ptr<E>(a.in, row), lo, hi,
                                 static_cast<E*>(a.grad) + (size_t)row * a.in.V + lo);
  Group<E> group;
  if (p.nvec) group = group_load<E, NT, ONCE>(p.vectors(), 0, p.nvec);
  const DistillStats st = a.stats[row];
  int id = -1;
  float q = 0.f;
  if ((int)tid < a.K) {
    const int64_t i = id_load(a.ids, a.in.rows, a.in.n, row, tid);
    if (i != a.ignore && i >= 0 && i < (int64_t)a.in.V) {
      id = (int)i;
      // (fp32, where the one call's q is fp64: four roundings leave the exponent
      // u <= 0 off by up to 2^-22 of itself, which moves q by at most
      // |u| e^u 2^-22 < 2^-23; an fp64 exponential would be each team's of a row.)
      q = __expf((list_load(a, row, tid) - st.tmax) * st.tscale) * st.qscale;
    }
  }
  if (tid < DistillLds<NT>::kList) {
    l.ids[tid] = id;
    l.q[tid] = q;
  }
  team_sync<NT>();
  distill_grad<E, NT, ONCE, 1, true>(a, row, p, st, id, l, &group);
}

// Groups of a row that stay in registers between its loss and its gradient: 64
// registers of a thread.  What is read again comes from the last-level cache
// and takes part of its bandwidth: 4096 rows of 131072 (bf16) take 525 us
// without, 455 with a quarter of the row held, by 256 threads; 451 with the
// same share by 512; 505 with the whole row by 1024, since then one row at a
// time has the CU and its loads, sums and stores follow one another.
template <typename E> constexpr int kHeld = 64 / ((int)sizeof(Group<E>) / 4);

template <typename E, bool TAIL, int NT, bool ONCE>
hipError_t distill_teams(DistillArgs a, bool grad, hipStream_t s) {
  const size_t lds = TAIL ? kTeams<NT> * bitmap_words<E>(a.split.len) * 4 : 0;
  return launch_items((uint64_t)a.in.rows * a.split.parts, kTeams<NT>,
                      [&](uint64_t first, uint32_t blocks) {
    a.first = first;
    TimedLaunch t(grad ? "distill_once" : "distill_rows", s);
    if (!grad)
      k_distill_rows<E, TAIL, false, 0, false, NT, ONCE><<<blocks, kTeamBlock<NT>, lds, s>>>(a);
    else if (NT == kWave || a.split.len <= NT * kGroup<E>)
      k_distill_rows<E, TAIL, true, 1, true, NT, ONCE><<<blocks, kTeamBlock<NT>, lds, s>>>(a);
    else if constexpr (NT > kWave) {
      constexpr int HG = kHeld<E>;
      if (a.split.len <= NT * kGroup<E> * HG)
        k_distill_rows<E, TAIL, true, HG, true, NT, ONCE><<<blocks, kTeamBlock<NT>, lds, s>>>(a);
      else
        k_distill_rows<E, TAIL, true, HG, false, NT, ONCE><<<blocks, kTeamBlock<NT>, lds, s>>>(a);
    }
  });
}

template <typename E, bool TAIL>
hipError_t distill_values(DistillArgs a, bool grad, hipStream_t s) {
  const bool once = read_once(a.in, sizeof(E));
  hipError_t e = a.split.nt == 64            ? distill_teams<E, TAIL, 64, false>(a, grad, s)
                 : a.split.nt == 256 && once ? distill_teams<E, TAIL, 256, true>(a, grad, s)
                 : a.split.nt == 256         ? distill_teams<E, TAIL, 256, false>(a, grad, s)
                 : once                      ? distill_teams<E, TAIL, 512, true>(a, grad, s)
                                             : distill_teams<E, TAIL, 512, false>(a, grad, s);
  if (e == hipSuccess && a.split.parts > 1)
    e = launch_items(a.in.rows, 1, [&](uint64_t first, uint32_t blocks) {
      a.first = first;
      TimedLaunch t("distill_join", s);
      k_distill_join<E, TAIL><<<blocks, 256, 0, s>>>(a);
    });
  return e;
}

template <typename E, int NT, bool ONCE>
hipError_t distill_grad_teams(DistillArgs a, hipStream_t s) {
  grad_chunks<E>(a.in.V, NT, &a.chunks, &a.len);
  return launch_items((uint64_t)a.in.rows * a.chunks, kTeams<NT>,
                      [&](uint64_t first, uint32_t blocks) {
    a.first = first;
    TimedLaunch t("distill_grad", s);
    k_distill_grad<E, NT, ONCE><<<blocks, kTeamBlock<NT>, 0, s>>>(a);
  });
}

template <typename E> hipError_t distill_gradient(const DistillArgs& a, hipStream_t s) {
  const bool wave = a.in.V <= kWave * kGroup<E> && a.in.rows >= 512 && a.K <= kListWave;
  return wave                         ? distill_grad_teams<E, 64, false>(a, s)
         : read_once(a.in, sizeof(E)) ? distill_grad_teams<E, 256, true>(a, s)
                                      : distill_grad_teams<E, 256, false>(a, s);
}

Split distill_split(int64_t rows, int64_t V, int K, int dtype, bool once) {
  // (Loss and gradient at once by a wave: of the one group it holds.)
  const int group = kWave * (dtype == SDTW_DTYPE_F32 ? kGroup<float> : kGroup<__bf16>);
  return split_rows(rows, V, K > kListWave ? 0 : once ? group : 4096);
}

size_t part_bytes(int64_t rows, const Split& sp) {
  return SDTW_ROWS_WORKSPACE_MIN +
         (sp.parts == 1 ? 0 : ((size_t)rows * sp.parts * sizeof(RowSums) + 255) / 256 * 256);
}

// Values first (values), then the gradient (grad not null).
template <typename E> int distill_run(DistillArgs a, bool tail, bool values, hipStream_t s) {
  const bool once = values && a.grad && a.split.parts == 1;
  hipError_t e = hipSuccess;
  if (values)
    e = tail ? distill_values<E, true>(a, once, s) : distill_values<E, false>(a, once, s);
  if (e == hipSuccess && a.grad && !once) e = distill_gradient<E>(a, s);
  return e == hipSuccess ? SDTW_OK : SDTW_ERR_HIP;
}

int distill_run(const DistillArgs& a, int dtype, bool tail, bool values, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return dtype == SDTW_DTYPE_F32    ? distill_run<float>(a, tail, values, s)
         : dtype == SDTW_DTYPE_BF16 ? distill_run<__bf16>(a, tail, values, s)
                                    : distill_run<_Float16>(a, tail, values, s);
}

}  // namespace
}  // namespace sdtw

extern "C" {

size_t sdtw_distill_workspace_bytes(int64_t B, int64_t N, int64_t V, int K) {
  using namespace sdtw;
  if (!rows_ok(B, N, V) || K < 1 || K > kListMax) return 0;
  return part_bytes(B * N, distill_split(B * N, V, K, SDTW_DTYPE_F32, false));
}

int sdtw_distill(const void* logits, int dtype, int64_t B, int64_t N, int64_t V, int64_t ld_b,
                 int64_t ld_n, const void* ids, int id_bytes, int64_t id_b, int64_t id_n,
                 const void* values, int value_dtype, int64_t val_b, int64_t val_n, int K,
                 int64_t ignore_index, double temperature, int tail, void* workspace,
                 size_t workspace_bytes, float* loss, float* stats, const float* grad_loss,
                 int64_t gl_step, void* grad_logits, void* stream) {
  using namespace sdtw;
  const size_t need = sdtw_distill_workspace_bytes(B, N, V, K);
  if (need == 0 || !temperature_ok(temperature) || !dtype_ok(dtype) || !dtype_ok(value_dtype) ||
      !logits || !ids || !values || (id_bytes != 4 && id_bytes != 8) || (!loss && !grad_logits) ||
      ((uintptr_t)stats & 15) || gl_step < 0 || gl_step > 1 || (tail != 0 && tail != 1))
    return SDTW_ERR_INVALID_ARG;
  DistillArgs a;
  a.in = rows_in(logits, B, N, V, ld_b, ld_n);
  a.split = distill_split(B * N, V, K, dtype, grad_logits != nullptr);
  // A gradient alone, or one from several launches, passes through `stats`.
  if (!stats && grad_logits && (!loss || a.split.parts > 1)) return SDTW_ERR_INVALID_ARG;
  if (loss) {
    if (((uintptr_t)workspace & 255) || (!workspace && need > SDTW_ROWS_WORKSPACE_MIN))
      return SDTW_ERR_INVALID_ARG;
    if (workspace_bytes < need) return SDTW_ERR_WORKSPACE;
  }
  a.ids = IdsIn{ids, id_b, id_n, id_bytes};
  a.list = IdsIn{values, val_b, val_n, value_dtype};
  a.ignore = ignore_index;
  a.c = make_scale(temperature);
  a.inv_t = 1.0 / temperature;
  a.K = K;
  a.part = static_cast<RowSums*>(workspace);
  a.loss = loss;
  a.stats = reinterpret_cast<DistillStats*>(stats);
  a.weight = grad_loss;
  a.w_step = gl_step;
  a.grad = grad_logits;
  return distill_run(a, dtype, tail != 0, loss != nullptr, stream);
}

}  // extern "C"
