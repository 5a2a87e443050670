// Entry points of the decoding operators (include/fg.h): argument checks and
// launches. Nothing is allocated or kept; every call is one or two kernels on
// the caller's stream, so all of them can be captured into a graph.
#include "fg_moe.hpp"
#include "fg_norm.hpp"
#include "fg_route.hpp"
#include "fg_w4.hpp"

using namespace fg::ops;

namespace {

// Launches on one stream, with their own errors only (an error that an earlier call
// of the program left behind is not theirs); none after one that failed.
struct Launches {
  hipStream_t stream;
  hipError_t error = hipSuccess;
  template <class Args>
  void operator()(void (*kernel)(Args), dim3 grid, dim3 block, size_t lds, Args a) {
    void* args[1] = {&a};
    if (error == hipSuccess) error = hipLaunchKernel((const void*)kernel, grid, block, args, lds, stream);
  }
  fg_status status() const { return error == hipSuccess ? FG_OK : FG_EHIP; }
};

constexpr int kCUs = 256;          // compute units of the part

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Rows of `bytes` bytes, `pitch` apart (one row: any pitch).
struct Rows {
  const void* p;
  int64_t rows, bytes, pitch;
  uintptr_t begin() const { return (uintptr_t)p; }
  uintptr_t end() const { return begin() + (rows - 1) * pitch + bytes; }
};
Rows whole(const void* p, int64_t bytes) { return {p, 1, bytes, bytes}; }

// Do they share a byte? Rows that interleave, as columns of one buffer do, need not.
bool overlap(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || a.end() <= b.begin() || b.end() <= a.begin()) return false;
  if (a.rows > b.rows) return overlap(b, a);
  if (a.pitch == b.pitch && a.rows > 1) {
    const int64_t d = (int64_t)(b.begin() - a.begin()) % a.pitch, shift = d < 0 ? d + a.pitch : d;
    if (shift >= a.bytes && shift + b.bytes <= a.pitch) return false;
  }
  for (int64_t i = 0; i < a.rows; ++i) {         // the last row of b that starts before the end of a's
    const uintptr_t from = a.begin() + i * a.pitch, to = from + a.bytes;
    if (to <= b.begin()) continue;
    const int64_t j = b.rows == 1 ? 0 : (int64_t)((to - 1 - b.begin()) / b.pitch);
    if (b.begin() + (j < b.rows ? j : b.rows - 1) * b.pitch + b.bytes > from) return true;
  }
  return false;
}
template <class... Others>
bool overlaps(const Rows& a, const Others&... others) { return (overlap(a, others) || ...); }

int pow2_at_least(int v) {
  int p = 1;
  while (p < v) p *= 2;
  return p;
}

// Activation rows of the products: whole 8-element vectors at aligned addresses.
bool rows_ok(const void* x, int64_t ldx, int32_t type, const float* scale, int32_t group, int32_t k) {
  if (!x || (type != FG_BF16 && type != FG_I8 && type != FG_E4M3)) return false;
  const int bytes = type == FG_BF16 ? 2 : 1;
  // a lane's distance from a tile's first row, up to 64 rows on, is 32 bits
  if (ldx < k || ldx % 8 || ldx * bytes >= FG_FEW_MAX_ROW_BYTES || !aligned(x, 8 * bytes)) return false;
  if (type == FG_BF16) return !scale && group == 0;
  return scale && aligned(scale, 4) && (group == 0 || (group == 128 && k % 128 == 0));
}

bool w4_ok(const void* w, const void* s, int32_t group, int32_t k) {
  return w && s && (group == 32 || group == 64 || group == 128) && k % group == 0 && aligned(w, 16) && aligned(s, 2);
}

// A grid of n workgroups for any n below 2^31: more than 2^20 in two dimensions
// (a dimension holds fewer than 2^32 threads).
dim3 wide_grid(int64_t n) {
  const int64_t x = 1 << 20;
  return n <= x ? dim3((unsigned)n) : dim3((unsigned)x, (unsigned)((n + x - 1) / x));
}

template <int W, int V>
void launch_norm(bool past, const NormArgs& a, Launches& go) {
  const dim3 grid = wide_grid((a.rows + NormShape<W>::kRows - 1) / NormShape<W>::kRows), block(NormShape<W>::kThreads);
  if (past) go(add_rmsnorm_kernel<W, V, true>, grid, block, 0, a);
  else go(add_rmsnorm_kernel<W, V, false>, grid, block, 0, a);
}

template <int W>
void launch_norm(int V, bool past, const NormArgs& a, Launches& go) {
  switch (V) {
    case 1: launch_norm<W, 1>(past, a, go); break;
    case 2: launch_norm<W, 2>(past, a, go); break;
    default:                       // more than two only where a row has all 16 waves
      if constexpr (W == 16) V == 4 ? launch_norm<W, 4>(past, a, go) : launch_norm<W, 8>(past, a, go);
  }
}

template <int L, int N, bool BF16>
void launch_route_lanes(const RouteArgs& a, Launches& go) {
  go(moe_route_kernel<L, N, BF16>, wide_grid((a.rows * L + 255) / 256), dim3(256), 0, a);
}

template <bool BF16>
void launch_route(const RouteArgs& a, Launches& go) {
  if (a.experts <= 16) launch_route_lanes<16, 1, BF16>(a, go);
  else if (a.experts <= 32) launch_route_lanes<16, 2, BF16>(a, go);
  else if (a.experts <= 64) launch_route_lanes<16, 4, BF16>(a, go);
  else if (a.experts <= 128) launch_route_lanes<16, 8, BF16>(a, go);
  else if (a.experts <= 256) launch_route_lanes<16, 16, BF16>(a, go);
  else if (a.experts <= 512) launch_route_lanes<64, 8, BF16>(a, go);
  else launch_route_lanes<64, 16, BF16>(a, go);
}

template <int G, int XK, int MT, int R, int P, int W>
void launch_w4_tile(const W4Args& a, Launches& go) {
  const dim3 grid((a.n + 16 * R - 1) / (16 * R), (a.rows + 16 * MT - 1) / (16 * MT));
  go(w4_linear_kernel<G, XK, MT, R, P, W>, grid, dim3(64 * W), XK == X_LDS ? 2 * (size_t)a.k : 0, a);
}

// The tile of 16 MT rows by 16 R columns. A larger one reads weights and
// activations fewer times, but a workgroup takes a compute unit's time whether or
// not the others have one: what counts is how many rounds of 256 workgroups there
// are, each as long as a tile's cost (measured at k = 4096 and 8192, in units of the
// smallest). Us for groups of 64, k = 8192, tiles (1,1) (1,2) (2,2) (4,2):
//               int8 rows            e4m3 rows
//   12 x 4096    7.7  9.7 12.0 16.0   8.3 11.0 13.6 17.7
//   12 x 8192   11.9 10.4 12.2 16.3  12.5 11.8 14.4 18.4
//   28 x 8192   18.4 16.2 12.2 16.3  19.8 18.2 14.5 18.4
//   60 x 4096   17.3 14.9 11.9 16.4  18.8 17.2 13.9 18.6
//   60 x 8192   32.7 27.6 20.3 17.4  35.0 31.4 23.1 19.6
// The largest does not fit in the registers for groups of 32.
// One row takes one of the first two.
template <int G, int XK>
void launch_w4(const W4Args& a, Launches& go) {
  constexpr int kTiles = XK == X_LDS ? 2 : G == 32 ? 3 : 4;
  auto rounds = [&](int mt, int r) {
    const int64_t n = (int64_t)((a.n + 16 * r - 1) / (16 * r)) * ((a.rows + 16 * mt - 1) / (16 * mt));
    return (n + kCUs - 1) / kCUs;
  };
  const float cost[4] = {1.0f * rounds(1, 1), 1.5f * rounds(1, 2), 2.2f * rounds(2, 2), 3.7f * rounds(4, 2)};
  int best = 0;
  for (int i = 1; i < kTiles; ++i)
    if (cost[i] < cost[best]) best = i;
  switch (best) {
    case 0:       // one workgroup or none a compute unit: more waves where they have enough steps (1 x 2048 x 7168: 5.6 us, with 8 5.9)
      if (rounds(1, 1) == 1 && a.k >= 48 * kStep) launch_w4_tile<G, XK, 1, 1, 2, 16>(a, go);
      else launch_w4_tile<G, XK, 1, 1, 2, 8>(a, go);
      break;
    case 1: launch_w4_tile<G, XK, 1, 2, 2, 8>(a, go); break;
    case 2:
      if constexpr (kTiles > 2) launch_w4_tile<G, XK, 2, 2, 1, 8>(a, go);
      break;
    default:
      if constexpr (kTiles > 3) launch_w4_tile<G, XK, 4, 2, 1, 8>(a, go);
  }
}

// One bf16 row goes through LDS: 1 x 2048 x 7168 5.6 us, straight from L2 6.3; 8192 x
// 8192 10.3 and 11.1; 4096 x 14336 9.0 and 10.6; with short rows there is no difference
// (64 x 512: 3.6). More rows would all be copied by every workgroup. Through LDS and
// from L2, at 4096 x 4096, 2048 x 7168 and 8192 x 4096: two rows 5.5 5.5, 6.1 6.4, 7.4
// 7.3 (4096 x 14336 10.0 11.2); three 5.8 5.6, 6.3 6.5, 7.7 7.4; four 6.0 5.5, 6.8 6.6,
// 7.9 7.4; eight 7.3 5.7, -, 9.0 7.3: two rows gain with long k alone, four lose. 8-bit
// rows have no such form. Rows of 32 KB leave room for the sums of the waves
// within 64 KB.
constexpr int kLdsRow = 16384;

template <int G>
void launch_w4(const W4Args& a, int type, bool grouped, Launches& go) {
  if (type == FG_BF16 && a.rows == 1 && a.k <= kLdsRow) launch_w4<G, X_LDS>(a, go);
  else if (type == FG_BF16) launch_w4<G, X_BF16>(a, go);
  else if (type == FG_I8) grouped ? launch_w4<G, X_I8G>(a, go) : launch_w4<G, X_I8>(a, go);
  else grouped ? launch_w4<G, X_E4M3G>(a, go) : launch_w4<G, X_E4M3>(a, go);
}

// More than 16 rows an expert on average, were all picks here: two row tiles, so
// that an expert's weights are still read once or twice; else one, whose fewer
// registers leave room for more waves. Us a layer with one and two row tiles, bf16
// weights, then 4-bit ones in groups of 128 with e4m3 rows and of 32 with int8 rows:
// 64 tokens over 64 experts of 7168 x 2048, 8 rows each: 4-bit e4m3 396 and 509; 8
// experts of that size, 32 rows each: 268 227, 126 131, int8 in groups of 64 129 128;
// 33 rows: 317 273, 144 154, 180 174; 64 rows: 410 322, 195 186, 242 209.
bool many_rows(const MoeArgs& a) { return a.tokens > 16 && a.tokens * a.k > 16 * a.n_local; }

template <int G, int XK, int MT, int C, int P, int W>
void launch_moe_up_tile(const MoeArgs& a, Launches& go) {
  const int picks = a.tokens * a.k, experts = picks < a.n_local ? picks : a.n_local;
  const dim3 grid(experts * ((a.F + 16 * C - 1) / (16 * C)));
  go(moe_up_kernel<G, XK, MT, C, P, W>, grid, dim3(64 * W), 0, a);
}

// 4-bit weights: two column tiles share the loads of x (a layer of 64 tokens over 64
// experts of 7168 x 2048, with two and with one: bf16 rows 394 and 410 us, int8 375 and
// 380, e4m3 390 and 392), where there are eight workgroups and more for each place on
// the compute units (15 tokens over 64 experts of 4480 x 1472: int8 89.4 and 88.6, e4m3
// 93.6 and 91.5); for groups of 32 they do not fit in the registers. Four waves: with
// eight, a workgroup's start and end are a larger share of it (12 tokens over 8 of 64 experts
// of 1792 x 1536: 7.6 us, with eight 8.9).
template <int G, int XK>
void launch_moe_up(const MoeArgs& a, Launches& go) {
  if constexpr (G == 0) {
    many_rows(a) ? launch_moe_up_tile<G, XK, 2, 1, 2, 4>(a, go) : launch_moe_up_tile<G, XK, 1, 1, 2, 4>(a, go);
  } else {
    const int picks = a.tokens * a.k;
    const int64_t pairs = (picks < a.n_local ? picks : a.n_local) * (int64_t)(a.F / 32);
    if (many_rows(a)) launch_moe_up_tile<G, XK, 2, 1, 1, 8>(a, go);
    else if (G == 32 || pairs < 16 * kCUs) launch_moe_up_tile<G, XK, 1, 1, 1, 4>(a, go);
    else if constexpr (G != 32) launch_moe_up_tile<G, XK, 1, 2, 1, 4>(a, go);
  }
}

template <int G, int MT, int R, int P, int W>
void launch_moe_down_tile(const MoeArgs& a, Launches& go) {
  const size_t lds = (size_t)W * a.tokens * 16 * R * sizeof(float);
  go(moe_down_kernel<G, MT, R, P, W>, dim3((a.K + 16 * R - 1) / (16 * R)), dim3(64 * W), lds, a);
}

// Two column tiles halve the reads of h (64 tokens over 64 experts: 167 us, with
// one 239 us), unless there are too few columns to give every second compute unit
// a workgroup then. Entries of up to 16 picks where an expert may have more than 8
// (one row tile there: 198 us; 16 tokens that all pick 8 experts of 928 x 672: 11.4
// us, with one row tile 12.2).
template <int G>
void launch_moe_down(const MoeArgs& a, Launches& go) {
  const bool few_columns = a.K < 32 * kCUs / 2;
  if (few_columns) a.tokens > 8 ? launch_moe_down_tile<G, 2, 1, 1, 8>(a, go) : launch_moe_down_tile<G, 1, 1, 1, 16>(a, go);
  else if (a.tokens > 16) launch_moe_down_tile<G, 2, 2, 2, 8>(a, go);
  else if constexpr (G == 0) launch_moe_down_tile<G, 1, 2, 1, 16>(a, go);
  else launch_moe_down_tile<G, 1, 2, 2, 8>(a, go);
}

template <int G>
fg_status launch_moe(const MoeArgs& a, int type, bool grouped, Launches& go) {
  if (type == FG_BF16) launch_moe_up<G, X_BF16>(a, go);
  else if (type == FG_I8) grouped ? launch_moe_up<G, X_I8G>(a, go) : launch_moe_up<G, X_I8>(a, go);
  else grouped ? launch_moe_up<G, X_E4M3G>(a, go) : launch_moe_up<G, X_E4M3>(a, go);
  launch_moe_down<G>(a, go);
  return go.status();
}

}  // namespace

extern "C" {

fg_status fg_add_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* gamma, float eps,
                         void* sum, int64_t lds, void* y, int64_t ldy, void* q, int64_t ldq, int32_t q_type,
                         int32_t q_group, float* q_scale, int64_t rows, int32_t n, hipStream_t stream) {
  if (rows < 0 || rows > 0x7fffffff || n < 1 || n > FG_NORM_MAX_N || !(eps >= 0.0f)) return FG_EINVAL;
  if (rows == 0) return FG_OK;
  if (!y && !q) return FG_EINVAL;
  if (q && ((q_type != FG_I8 && q_type != FG_E4M3) || !q_scale || (q_group != 0 && (q_group != 128 || n % 128)))) return FG_EINVAL;
  if (!x || !gamma || ldx < n || (residual && ldr < n) || (sum && lds < n) || (y && ldy < n) || (q && ldq < n)) return FG_EINVAL;
  if (!aligned(x, 2) || !aligned(residual, 2) || !aligned(gamma, 2) || !aligned(sum, 2) || !aligned(y, 2) || !aligned(q_scale, 4))
    return FG_EINVAL;
  Launches go{stream};
  NormArgs a{};
  a.x = (const uint16_t*)x; a.res = (const uint16_t*)residual; a.gamma = (const uint16_t*)gamma;
  a.sum = (uint16_t*)sum; a.y = (uint16_t*)y; a.q = (uint8_t*)q; a.scale = q_scale;
  a.ldx = ldx; a.ldr = ldr; a.lds = lds; a.ldy = ldy; a.ldq = ldq; a.rows = rows;
  a.n = n; a.group = q ? q_group : 0; a.q_type = q_type; a.eps = eps;
  // Few rows: as many threads a row as it takes, for the latency. Many: 16 elements
  // a thread, and stores past the caches once the outputs exceed them (8192 x 7168,
  // residual, e4m3: 80 us; with 8 and 32 elements a thread 85 and 84 us; with
  // ordinary stores 82 us).
  const bool past = rows * n > ((int64_t)32 << 20) / 2;
  const int nv = (n + 7) / 8, want = rows < 1024 ? 1 : 2;
  int W = pow2_at_least((nv + 64 * want - 1) / (64 * want));
  if (W > 16) W = 16;
  const int V = pow2_at_least((nv + 64 * W - 1) / (64 * W));
  switch (W) {
    case 1: launch_norm<1>(V, past, a, go); break;
    case 2: launch_norm<2>(V, past, a, go); break;
    case 4: launch_norm<4>(V, past, a, go); break;
    case 8: launch_norm<8>(V, past, a, go); break;
    default: launch_norm<16>(V, past, a, go); break;
  }
  return go.status();
}

fg_status fg_moe_route(const void* logits, int64_t ld, int32_t logits_type, int64_t rows, int32_t experts, int32_t k,
                       int32_t score, int32_t renorm, float scale, int32_t* topk, float* weights, hipStream_t stream) {
  if (rows < 0 || rows > 0x7fffffff || experts < 1 || experts > FG_MOE_FEW_EXPERTS || k < 1 || k > experts || k > 64) return FG_EINVAL;
  if ((logits_type != FG_F32 && logits_type != FG_BF16) || (score != FG_SCORE_SOFTMAX && score != FG_SCORE_SIGMOID)) return FG_EINVAL;
  if (rows == 0) return FG_OK;
  if (!logits || !topk || !weights || ld < experts) return FG_EINVAL;
  if (!aligned(logits, logits_type == FG_F32 ? 4 : 2) || !aligned(topk, 4) || !aligned(weights, 4)) return FG_EINVAL;
  const int64_t element = logits_type == FG_F32 ? 4 : 2;
  const Rows in{logits, rows, element * experts, element * ld}, picks = whole(topk, 4 * rows * k), gates = whole(weights, 4 * rows * k);
  if (overlaps(picks, in, gates) || overlaps(gates, in)) return FG_EINVAL;
  Launches go{stream};
  RouteArgs a{logits, topk, weights, ld, rows, experts, k, score, renorm, scale};
  logits_type == FG_BF16 ? launch_route<true>(a, go) : launch_route<false>(a, go);
  return go.status();
}

fg_status fg_w4_linear(const void* x, int64_t ldx, int32_t x_type, const float* x_scale, int32_t x_group, const void* w,
                       const void* w_scale, const void* w_zero, int32_t group, const void* bias, void* out, int64_t ldo,
                       int64_t rows, int32_t n, int32_t k, hipStream_t stream) {
  if (rows < 0 || rows > FG_W4_MAX_ROWS || n < 1 || k < 1 || n > FG_FEW_MAX_SIZE || k > FG_FEW_MAX_SIZE || !w4_ok(w, w_scale, group, k)) return FG_EINVAL;
  if (rows == 0) return FG_OK;
  if (!rows_ok(x, ldx, x_type, x_scale, x_group, k) || !out || ldo < n || !aligned(out, 2) || !aligned(bias, 2)) return FG_EINVAL;
  const int64_t element = x_type == FG_BF16 ? 2 : 1, groups = k / group;
  // workgroups write their columns while others still read
  if (overlaps(Rows{out, rows, 2 * (int64_t)n, 2 * ldo}, Rows{x, rows, element * k, element * ldx},
               whole(x_scale, 4 * rows * (x_group ? k / x_group : 1)), whole(w, (int64_t)n * k / 2), whole(w_scale, 2 * n * groups),
               whole(w_zero, n * groups), whole(bias, 2 * (int64_t)n)))
    return FG_EINVAL;
  Launches go{stream};
  W4Args a{};
  a.x = (const char*)x; a.xs = x_scale; a.w = (const char*)w; a.s = (const uint16_t*)w_scale; a.z = (const uint8_t*)w_zero;
  a.bias = (const uint16_t*)bias; a.out = (uint16_t*)out;
  a.ldx = ldx * (x_type == FG_BF16 ? 2 : 1); a.xs_stride = x_group ? k / x_group : 1; a.ldo = ldo;
  a.rows = (int32_t)rows; a.n = n; a.k = k;
  if (group == 32) launch_w4<32>(a, x_type, x_group != 0, go);
  else if (group == 64) launch_w4<64>(a, x_type, x_group != 0, go);
  else launch_w4<128>(a, x_type, x_group != 0, go);
  return go.status();
}

fg_status fg_moe_few_bytes(int32_t tokens, int32_t k, int32_t F, int64_t* bytes) {
  if (!bytes || tokens < 0 || tokens > FG_MOE_FEW_TOKENS || k < 1 || k > FG_MOE_FEW_TOPK || F < 1) return FG_EINVAL;
  *bytes = 4 * (int64_t)tokens * k * F;
  return FG_OK;
}

fg_status fg_moe_few(const void* x, int64_t ldx, int32_t x_type, const float* x_scale, int32_t x_group, const void* w1,
                     const void* w1_scale, const void* w1_zero, const void* w2, const void* w2_scale, const void* w2_zero,
                     int32_t group, const int32_t* topk, const float* weights, int32_t tokens, int32_t k,
                     int32_t expert_base, int32_t n_local, int32_t K, int32_t F, void* workspace, int64_t workspace_bytes,
                     void* y, int64_t ldy, hipStream_t stream) {
  if (tokens < 0 || tokens > FG_MOE_FEW_TOKENS || k < 1 || k > FG_MOE_FEW_TOPK || n_local < 1 || n_local > FG_MOE_FEW_EXPERTS ||
      expert_base < 0 || expert_base > 0x7fffffff - FG_MOE_FEW_EXPERTS || K < 1 || F < 1 || K > FG_FEW_MAX_SIZE || F > FG_FEW_MAX_SIZE || K % 32 || F % 32)
    return FG_EINVAL;
  // the distance from a gate row to its up row, in bytes, is 32 bits
  if (((int64_t)F + 32) * K * (group ? 1 : 4) / 2 > 0xffffffff) return FG_EINVAL;
  if (group == 0) {
    if (!w1 || !w2 || w1_scale || w2_scale || w1_zero || w2_zero || !aligned(w1, 16) || !aligned(w2, 16)) return FG_EINVAL;
  } else if (!w4_ok(w1, w1_scale, group, K) || !w4_ok(w2, w2_scale, group, F)) {
    return FG_EINVAL;
  }
  if (tokens == 0) return FG_OK;
  if (!rows_ok(x, ldx, x_type, x_scale, x_group, K) || !topk || !weights || !y || ldy < K) return FG_EINVAL;
  if (!aligned(topk, 4) || !aligned(weights, 4) || !aligned(y, 2)) return FG_EINVAL;
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < 4 * (int64_t)tokens * k * F) return FG_EINVAL;
  {
    // the first kernel reads all but w2 and writes the workspace, the second reads w2, topk and the workspace and writes y
    const int64_t element = x_type == FG_BF16 ? 2 : 1, elements = (int64_t)n_local * K * F, per = group ? group : 1, picks = 4 * (int64_t)tokens * k;
    const int64_t bytes = group ? elements / 2 : 2 * elements;
    const Rows h = whole(workspace, picks * F), sum{y, tokens, 2 * (int64_t)K, 2 * ldy}, ids = whole(topk, picks);
    const Rows b = whole(w2, bytes), sb = whole(w2_scale, 2 * elements / per), zb = whole(w2_zero, elements / per);
    if (overlaps(h, ids, sum, b, sb, zb, Rows{x, tokens, element * K, element * ldx}, whole(x_scale, 4 * (int64_t)tokens * (x_group ? K / x_group : 1)),
                 whole(weights, picks), whole(w1, 2 * bytes), whole(w1_scale, 4 * elements / per), whole(w1_zero, 2 * elements / per)) ||
        overlaps(sum, ids, b, sb, zb))
      return FG_EINVAL;
  }
  Launches go{stream};
  MoeArgs a{};
  a.x = (const char*)x; a.xs = x_scale; a.topk = topk; a.weights = weights;
  a.w1 = (const char*)w1; a.s1 = (const uint16_t*)w1_scale; a.z1 = (const uint8_t*)w1_zero;
  a.w2 = (const char*)w2; a.s2 = (const uint16_t*)w2_scale; a.z2 = (const uint8_t*)w2_zero;
  a.h = (char*)workspace; a.plane = 32 * (uint32_t)(tokens * k);
  a.y = (uint16_t*)y;
  a.ldx = ldx * (x_type == FG_BF16 ? 2 : 1); a.xs_stride = x_group ? K / x_group : 1; a.ldy = ldy;
  a.tokens = tokens; a.k = k; a.base = expert_base; a.n_local = n_local; a.K = K; a.F = F;
  // a grid of fewer than 2^32 threads: the first product's workgroups have 256, those of 4-bit weights and many rows 512
  const int64_t workgroups = (int64_t)n_local * ((F + 15) / 16);
  if (workgroups > 1 << 23 || (workgroups == 1 << 23 && group && many_rows(a))) return FG_EINVAL;
  const bool grouped = x_group != 0;
  if (group == 0) return launch_moe<0>(a, x_type, grouped, go);
  if (group == 32) return launch_moe<32>(a, x_type, grouped, go);
  if (group == 64) return launch_moe<64>(a, x_type, grouped, go);
  return launch_moe<128>(a, x_type, grouped, go);
}

}  // extern "C"
