// Log-probabilities of given tokens with the entropy and the top alternatives
// of each row, and their gradient (sdtw_token_* of include/sdtw.h).
//
// Over a row of logits, with t_j = z_j log2(e) / T less a reference near the
// largest of them:
//   S = sum 2^t_j,  W = sum 2^t_j t_j,
//   log p_j = ln2 (t_j - log2 S),  H = ln2 (log2 S - W / S),
// so one pass gives every statistic, and the gradient pass needs no more of
// the forward than the reference, S and H:
//   dz_j = (1/T) [ g d_(j,token) + sum_i G_i d_(j,top_i)
//                  - p_j (g + sum_i G_i + gH (log p_j + H)) ].
#include "sdtw.h"
#include "sdtw_kernels.h"
#include "sdtw_rows.h"

namespace sdtw {
namespace {

struct TokenArgs {
  RowsIn in;
  uint64_t first;          // item of the launch's first team
  IdsIn tokens;            // p null: no given tokens
  int64_t ignore;
  float c;
  int k;                   // top entries (0: none)
  Split split;
  RowSums* part;           // [rows, parts] (parts > 1)
  uint64_t* part_keys;     // [rows, parts, k]
  float* logprob;          // [rows]
  float* entropy;          // [rows]
  float4* stats;           // [rows] what the backward needs, or null
  float* top_logprob;      // [rows, k]
  int64_t* top_token;      // [rows, k]
};

// Results of a row from its statistics and (k > 0) its top keys, by a team.
template <typename E, int NT>
__device__ __forceinline__ void token_finish(const TokenArgs& a, uint32_t row, const RowSums& r,
                                             const uint64_t* best) {
  const bool none = r.s == 0.0 && r.m == -__builtin_inff();
  const Exponent x = row_exponent(r.m, a.c);
  const double ln_s = none ? 0.0 : ln32(r.s);
  // A row without any entry above -inf gives every token probability zero.  An
  // entry with all of the probability has an exponent that is what the rounding
  // of the reference left, and an S whose exponential and logarithm are rounded:
  // they cancel to 1e-7, on either side of zero.  (A NaN stays one.)
  auto logprob_of = [&](float z) {
    const float lp = none ? -__builtin_inff() : (float)(kLn2 * exponent64(x, z) - ln_s);
    return lp > 0.f ? 0.f : lp;
  };
  const int tid = team_tid<NT>();
  if (tid == 0) {
    // The logits' NaN, or a maximum of +inf, has made S a NaN.
    const double h = none ? 0.0 : ln_s - kLn2 * (r.w / r.s);
    a.entropy[row] = h < 0.0 ? 0.f : (float)h;
    if (a.stats) {
      const float inv_s = none ? 0.f : (float)(1.0 / r.s);
      a.stats[row] = make_float4(x.ref, inv_s, (float)(h - ln_s), x.far ? 1.f : 0.f);
    }
    if (a.tokens.p) {
      const int64_t t = id_load(a.tokens, a.in.rows, a.in.n, row, 0);
      float lp = __builtin_nanf("");
      if (t == a.ignore) lp = 0.f;
      else if (t >= 0 && t < (int64_t)a.in.V) lp = logprob_of((float)row_ptr<E>(a.in, row)[t]);
      a.logprob[row] = lp;
    }
  }
  for (int i = tid; i < a.k; i += NT) {
    const uint64_t key = best[i];
    a.top_token[(size_t)row * a.k + i] = (int64_t)key_index(key);
    a.top_logprob[(size_t)row * a.k + i] =
        __builtin_isnan(r.s) ? __builtin_nanf("") : logprob_of(key_value(key));
  }
}

// One part of a row per team, read once; the row's results where it is whole.
// Each entry takes a conversion, a maximum, an fma, an exponential (two issue
// slots), a sum and an fma for W: bound by memory where 16-bit rows come from
// HBM, and within a tenth by issue.  4096 rows of 131072 (bf16): 165 us, 6.5
// TB/s (157 us, 6.8, at its best); with the top 64 of
// each 2048: 112 us, 4.8 TB/s; 1024 rows of 65537 (fp16, in the last-level
// cache) with the top 5: 34 us.  One row of 32768 with the top 20: 11 us, of
// which 6 are the launch as events see it: the chain of one row's read, its
// bound, its candidates' second read and their ranks.
template <typename E, bool TOP, int NT, bool ONCE> __global__ __launch_bounds__(kTeamBlock<NT>) void
k_token_rows(TokenArgs a) {
  __shared__ ReduceLds<NT> red;          // (a wave reduces in registers)
  __shared__ TopLds<NT> tops[TOP ? kTeams<NT> : 1];
  extern __shared__ float gmaxes[];      // TOP: [teams][groups][NT]
  TopLds<NT>& top = tops[TOP ? team_id<NT>() : 0];
  float* gmax = TOP ? gmaxes + team_id<NT>() * (gmax_bytes<E, NT>(a.split.len) / 4) : nullptr;
  const uint64_t items = (uint64_t)a.in.rows * a.split.parts;
  const uint64_t item = a.first + (uint64_t)blockIdx.x * kTeams<NT> + team_id<NT>();
  if (item >= items) return;
  const uint32_t row = a.split.parts == 1 ? (uint32_t)item : (uint32_t)(item / a.split.parts);
  const uint32_t lo = (uint32_t)(item - (uint64_t)row * a.split.parts) * a.split.len;
  const uint32_t hi = min(a.in.V, lo + a.split.len);
  const E* z = row_ptr<E>(a.in, row);
  const Part<E> p = make_part<E>(z, lo, hi, z + lo);
  auto start = row_start<E, NT, ONCE, 0, false>(p);
  float mine;
  const RowSums r =
      part_sums<E, NT, true, false, ONCE, 0, false>(p, a.c, nullptr, gmax, start, mine, red);
  if (TOP) {
    // Threads beyond the part's vectors and other entries have none.
    const uint32_t tid = team_tid<NT>();
    const bool has = tid < p.nvec || tid < p.rests();
    const int k = min(a.k, (int)p.len);
    if (k < a.k) {
      // A part shorter than k: the missing keys are zero, below every other.
      for (int i = tid; i < a.k; i += NT) top.best[i] = 0;
      team_sync<NT>();
    }
    top_entries<E, NT>(p, gmax, has ? value_order(mine) : 0u, k, top);
  }
  if (a.split.parts == 1) {
    token_finish<E, NT>(a, row, r, TOP ? top.best : nullptr);
  } else {
    if (team_tid<NT>() == 0) a.part[item] = r;
    if (TOP)
      for (int i = team_tid<NT>(); i < a.k; i += NT) a.part_keys[item * a.k + i] = top.best[i];
  }
}

// Joins the parts of a row: a block a row, bound by latency (0.6 us more for one
// row of 131072 in parts than for the same row whole).
template <typename E, bool TOP> __global__ __launch_bounds__(256) void k_token_join(TokenArgs a) {
  constexpr int NT = 256;
  __shared__ ReduceLds<NT> red;
  __shared__ TopLds<NT> top;
  const uint32_t row = (uint32_t)a.first + blockIdx.x;
  RowSums mine{-__builtin_inff(), 0.0, 0.0};
  for (uint32_t i = threadIdx.x; i < a.split.parts; i += NT)
    sums_join<true>(mine, a.part[(size_t)row * a.split.parts + i], a.c);
  const RowSums r = team_join<NT, true>(mine, a.c, red);
  if (TOP) {
    const uint32_t n = a.split.parts * (uint32_t)a.k;
    top_of_keys<NT>(a.part_keys + (size_t)row * n, n, a.k, top);
  }
  token_finish<E, NT>(a, row, r, TOP ? top.best : nullptr);
}

struct TokenGradArgs {
  RowsIn in;
  uint64_t first;            // item of the launch's first team
  IdsIn tokens;
  int64_t ignore;
  float c, inv_t;
  int k;
  uint32_t chunks, len;      // teams of a row, entries of each
  const float4* stats;
  const int64_t* top_token;  // [rows, k]
  const float* g_logprob;    // one a row, gl_step apart (0: one for all), or null
  const float* g_entropy;
  const float* g_top;        // [rows, k] or null
  int64_t gl_step, ge_step;
  void* grad;                // [rows, V]
};

// One team writes one group of a row, whose loads are asked for before the row's
// statistics: no loop, and as many blocks as the GPU holds are at different
// points of it.  Bound by memory, one read and one write: 4096 rows of 131072
// (bf16) take 345 us, 6.2 TB/s (torch's copy: 4.9).
template <typename E, int NT, bool ONCE> __global__ __launch_bounds__(256) void
k_token_grad(TokenGradArgs a) {
  constexpr int n = kRowVec<E>, U = kRowUnroll<E>;
  __shared__ ReduceLds<NT> red;
  const uint32_t tid = team_tid<NT>();
  const uint64_t items = (uint64_t)a.in.rows * a.chunks;
  const uint64_t item = a.first + (uint64_t)blockIdx.x * kTeams<NT> + team_id<NT>();
  if (item >= items) return;
  const uint32_t row = a.chunks == 1 ? (uint32_t)item : (uint32_t)(item / a.chunks);
  const uint32_t lo = (uint32_t)(item - (uint64_t)row * a.chunks) * a.len;
  const uint32_t hi = min(a.in.V, lo + a.len);
  E* out = static_cast<E*>(a.grad) + (size_t)row * a.in.V + lo;
  const Part<E> part = make_part<E>(row_ptr<E>(a.in, row), lo, hi, out);
  const E* z = part.z;
  Group<E> group;
  if (part.nvec) group = group_load<E, NT, ONCE>(part.vectors(), 0, part.nvec);
  const float4 st = a.stats[row];
  const Exponent ex{a.c, st.x, st.w != 0.f};
  const bool none = st.y == 0.f;
  int64_t token = a.ignore;
  float g = 0.f;
  if (a.g_logprob) {
    token = id_load(a.tokens, a.in.rows, a.in.n, row, 0);
    if (token != a.ignore) {
      g = a.g_logprob[(size_t)row * a.gl_step];
      if (token < 0 || token >= (int64_t)a.in.V) g = __builtin_nanf("");
    }
  }
  const float gh = a.g_entropy ? a.g_entropy[(size_t)row * a.ge_step] : 0.f;
  float sum = 0.f;
  if (a.g_top) {
    double part = 0.0;
    for (int i = tid; i < a.k; i += NT) part += (double)a.g_top[(size_t)row * a.k + i];
    sum = (float)team_sum<NT>(part, red);
  }
  // dz = e (A + B t) with e = 2^t
  const float B = -gh * st.y * a.inv_t * (float)kLn2;
  const float A = -(g + sum + gh * st.z) * st.y * a.inv_t;
  const bool zero = none || (g == 0.f && sum == 0.f && gh == 0.f);
  // A row without a distribution, or without an upstream gradient: zero.
  // (Gradients of top entries that cancel are none.)
  auto write = [&](auto value) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t v = u * NT + tid;
      auto x = row_wide<E>(group.v[u]);
#pragma unroll
      for (int i = 0; i < n; ++i) x[i] = value(x[i]);
      if (v < part.nvec) row_store<E, ONCE>(out + part.head + (size_t)v * n, x);
    }
    const uint32_t rest = part.rest(tid);
    if (rest < part.len) out[rest] = (E)value((float)z[rest]);
  };
  auto one = [&](float x, auto far) {
    const float t = exponent<decltype(far)::value>(ex, x);
    return hw_exp2(t) * __builtin_fmaf(B, fmaxf(t, -200.f), A);
  };
  if (zero) write([](float) { return 0.f; });
  else if (ex.far) write([&](float x) { return one(x, std::true_type()); });
  else if (B == 0.f) write([&](float x) { return hw_exp2(exponent<false>(ex, x)) * A; });
  else write([&](float x) { return one(x, std::false_type()); });
  team_sync<NT>();
  if (!none) {
    // The given token and the top entries have terms of their own; each is
    // written by one thread, behind the others.
    auto special = [&](int64_t id, float term) {
      if (id >= lo && id < hi) {
        const float x = (float)z[id - lo];
        const float p = zero ? 0.f : ex.far ? one(x, std::true_type()) : one(x, std::false_type());
        out[id - lo] = (E)__builtin_fmaf(a.inv_t, term, p);
      }
    };
    bool met = false;
    if (a.g_top)
      for (int i = tid; i < a.k; i += NT) {
        const int64_t id = a.top_token[(size_t)row * a.k + i];
        met |= id == token;
        special(id, a.g_top[(size_t)row * a.k + i] + (id == token ? g : 0.f));
      }
    if (a.g_top) {
      team_sync<NT>();
      met = team_sum<NT>(met ? 1.0 : 0.0, red) != 0.0;
    }
    if (tid == NT - 1 && !met && g != 0.f) special(token, g);
  }
}

template <typename E, int NT, bool ONCE>
hipError_t token_rows_launch(TokenArgs a, hipStream_t s) {
  const size_t lds = kTeams<NT> * gmax_bytes<E, NT>(a.split.len);
  return launch_items((uint64_t)a.in.rows * a.split.parts, kTeams<NT>,
                      [&](uint64_t first, uint32_t blocks) {
    a.first = first;
    TimedLaunch t("token_rows", s);
    if (a.k) k_token_rows<E, true, NT, ONCE><<<blocks, kTeamBlock<NT>, lds, s>>>(a);
    else k_token_rows<E, false, NT, ONCE><<<blocks, kTeamBlock<NT>, 0, s>>>(a);
  });
}

template <typename E> hipError_t token_launch(TokenArgs a, hipStream_t s) {
  const bool once = read_once(a.in, sizeof(E));
  hipError_t e = a.split.nt == 64            ? token_rows_launch<E, 64, false>(a, s)
                 : a.split.nt == 256 && once ? token_rows_launch<E, 256, true>(a, s)
                 : a.split.nt == 256         ? token_rows_launch<E, 256, false>(a, s)
                 : once                      ? token_rows_launch<E, 512, true>(a, s)
                                             : token_rows_launch<E, 512, false>(a, s);
  if (e == hipSuccess && a.split.parts > 1)
    e = launch_items(a.in.rows, 1, [&](uint64_t first, uint32_t blocks) {
      a.first = first;
      TimedLaunch t("token_join", s);
      if (a.k) k_token_join<E, true><<<blocks, 256, 0, s>>>(a);
      else k_token_join<E, false><<<blocks, 256, 0, s>>>(a);
    });
  return e;
}

template <typename E, int NT, bool ONCE>
hipError_t token_grad_teams(TokenGradArgs a, hipStream_t s) {
  grad_chunks<E>(a.in.V, NT, &a.chunks, &a.len);
  return launch_items((uint64_t)a.in.rows * a.chunks, kTeams<NT>,
                      [&](uint64_t first, uint32_t blocks) {
    a.first = first;
    TimedLaunch t("token_grad", s);
    k_token_grad<E, NT, ONCE><<<blocks, kTeamBlock<NT>, 0, s>>>(a);
  });
}

template <typename E> hipError_t token_grad_launch(const TokenGradArgs& a, hipStream_t s) {
  return a.in.V <= kWave * kGroup<E> && a.in.rows >= 512 ? token_grad_teams<E, 64, false>(a, s)
         : read_once(a.in, sizeof(E))       ? token_grad_teams<E, 256, true>(a, s)
                                            : token_grad_teams<E, 256, false>(a, s);
}

Split token_split(int64_t rows, int64_t V, int k) {
  // (256: all the entries may be candidates of a team of one wave.)
  return split_rows(rows, V, k <= kTopWave ? 4096 : 256);
}

size_t token_workspace(int64_t rows, int64_t V, int k) {
  const Split sp = token_split(rows, V, k);
  if (sp.parts == 1) return SDTW_ROWS_WORKSPACE_MIN;
  const size_t n = (size_t)rows * sp.parts;
  return SDTW_ROWS_WORKSPACE_MIN + (n * sizeof(RowSums) + n * (size_t)k * 8 + 255) / 256 * 256;
}

bool ids_ok(const void* p, int bytes) { return p == nullptr || bytes == 4 || bytes == 8; }

}  // namespace
}  // namespace sdtw

extern "C" {

size_t sdtw_token_workspace_bytes(int64_t B, int64_t N, int64_t V, int top_k) {
  if (!sdtw::rows_ok(B, N, V) || top_k < 0 || top_k > sdtw::kTopMax || top_k > V) return 0;
  return sdtw::token_workspace(B * N, V, top_k);
}

int sdtw_token_logprobs(const void* logits, int dtype, int64_t B, int64_t N, int64_t V,
                        int64_t ld_b, int64_t ld_n, const void* tokens, int token_bytes,
                        int64_t tok_b, int64_t tok_n, int64_t ignore_index, double temperature,
                        int top_k, void* workspace, size_t workspace_bytes, float* logprobs,
                        float* entropy, float* stats, float* top_logprobs, int64_t* top_tokens,
                        void* stream) {
  using namespace sdtw;
  const size_t need = sdtw_token_workspace_bytes(B, N, V, top_k);
  if (need == 0 || !temperature_ok(temperature) || !dtype_ok(dtype) || !logits || !entropy ||
      !ids_ok(tokens, token_bytes) || (tokens && !logprobs) ||
      (top_k && (!top_logprobs || !top_tokens)) || ((uintptr_t)stats & 15))
    return SDTW_ERR_INVALID_ARG;
  if (((uintptr_t)workspace & 255) || (!workspace && need > SDTW_ROWS_WORKSPACE_MIN))
    return SDTW_ERR_INVALID_ARG;
  if (workspace_bytes < need) return SDTW_ERR_WORKSPACE;
  TokenArgs a;
  a.in = rows_in(logits, B, N, V, ld_b, ld_n);
  a.tokens = IdsIn{tokens, tok_b, tok_n, token_bytes};
  a.ignore = ignore_index;
  a.c = make_scale(temperature);
  a.k = top_k;
  a.split = token_split(B * N, V, top_k);
  a.part = static_cast<RowSums*>(workspace);
  a.part_keys = reinterpret_cast<uint64_t*>(a.part + (size_t)a.in.rows * a.split.parts);
  a.logprob = logprobs;
  a.entropy = entropy;
  a.stats = reinterpret_cast<float4*>(stats);
  a.top_logprob = top_logprobs;
  a.top_token = top_tokens;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = dtype == SDTW_DTYPE_F32    ? token_launch<float>(a, s)
                       : dtype == SDTW_DTYPE_BF16 ? token_launch<__bf16>(a, s)
                                                  : token_launch<_Float16>(a, s);
  return e == hipSuccess ? SDTW_OK : SDTW_ERR_HIP;
}

int sdtw_token_backward(const void* logits, int dtype, int64_t B, int64_t N, int64_t V,
                        int64_t ld_b, int64_t ld_n, const void* tokens, int token_bytes,
                        int64_t tok_b, int64_t tok_n, int64_t ignore_index, double temperature,
                        int top_k, const float* stats, const int64_t* top_tokens,
                        const float* grad_logprobs, int64_t gl_step, const float* grad_entropy,
                        int64_t ge_step, const float* grad_top, void* grad_logits, void* stream) {
  using namespace sdtw;
  if (!rows_ok(B, N, V) || top_k < 0 || top_k > kTopMax || top_k > V ||
      !temperature_ok(temperature) || !dtype_ok(dtype) || !logits || !stats || !grad_logits ||
      ((uintptr_t)stats & 15) || !ids_ok(tokens, token_bytes) || (grad_logprobs && !tokens) ||
      (grad_top && (top_k == 0 || !top_tokens)) || gl_step < 0 || gl_step > 1 || ge_step < 0 ||
      ge_step > 1)
    return SDTW_ERR_INVALID_ARG;
  TokenGradArgs a;
  a.in = rows_in(logits, B, N, V, ld_b, ld_n);
  a.tokens = IdsIn{tokens, tok_b, tok_n, token_bytes};
  a.ignore = ignore_index;
  a.c = make_scale(temperature);
  a.inv_t = (float)(1.0 / temperature);
  a.k = top_k;
  a.stats = reinterpret_cast<const float4*>(stats);
  a.top_token = top_tokens;
  a.g_logprob = grad_logprobs;
  a.gl_step = gl_step;
  a.g_entropy = grad_entropy;
  a.ge_step = ge_step;
  a.g_top = grad_top;
  a.grad = grad_logits;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = dtype == SDTW_DTYPE_F32    ? token_grad_launch<float>(a, s)
                       : dtype == SDTW_DTYPE_BF16 ? token_grad_launch<__bf16>(a, s)
                                                  : token_grad_launch<_Float16>(a, s);
  return e == hipSuccess ? SDTW_OK : SDTW_ERR_HIP;
}

}  // extern "C"
