// C-ABI entry points of the layer operators (products with an epilogue, norms, their backward
// passes, quantised rows): argument validation, planning and launch.  Every check runs before any HIP call.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <string>

#include "ep.h"
#include "norm.h"
#include "tg_internal.h"

using namespace tg;

namespace {

const int64_t kMaxDim = (int64_t)1 << 30;
const int64_t kMaxIntK = 131071;                 // 128·128·K stays below 2^31
const int64_t kMaxLd = (int64_t)1 << 40;
const int64_t kMaxSpan = (int64_t)1 << 60;      // elements from a matrix's first row to its last
const int64_t kDirectSpan = (int64_t)1 << 31;   // buffer offsets of the direct loads stay below

std::string fmt(const char* f, long long a = 0, long long b = 0, long long c = 0) {
  char buf[256];
  std::snprintf(buf, sizeof buf, f, a, b, c);
  return buf;
}

bool is16(int t) { return t == TG_F16 || t == TG_BF16; }
bool isf8(int t) { return t == TG_FP8_E4M3 || t == TG_FP8_E5M2; }
bool is8(int t) { return isf8(t) || t == TG_I8; }
bool is_float(int t) { return is16(t) || t == TG_F32; }
int bytes_of(int t) { return t == TG_F32 ? 4 : is16(t) ? 2 : 1; }

// A matrix argument: `rows` runs of `width` bytes, `pitch` bytes apart.
struct Mat {
  const void* p;
  int64_t rows, width, pitch;
};
Mat mat(const void* p, int64_t rows, int64_t cols, int64_t ld, int eb) {
  return Mat{p, rows, cols * eb, ld * eb};
}
Mat vec(const void* p, int64_t n, int eb) { return Mat{p, 1, n * eb, n * eb}; }

bool overlaps(const Mat& a, const Mat& b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  const uintptr_t a1 = a0 + (uintptr_t)((a.rows - 1) * a.pitch + a.width);
  const uintptr_t b1 = b0 + (uintptr_t)((b.rows - 1) * b.pitch + b.width);
  if (!(a0 < b1 && b0 < a1)) return false;
  if (a.pitch != b.pitch) return true;
  // same row pitch: disjoint when b's columns lie in the gap behind a's
  const int64_t p = a.pitch;
  const int64_t d = (((int64_t)(b0 - a0)) % p + p) % p;
  return !(d >= a.width && d + b.width <= p);
}
bool same(const Mat& a, const Mat& b) { return a.p == b.p && a.pitch == b.pitch; }

// ld 0 = packed; must cover the row, and the rows must lie in an address space: byte spans stay below 2^63
int resolve_ld(const char* name, int64_t* ld, int64_t cols, int64_t rows) {
  if (*ld == 0) *ld = std::max<int64_t>(cols, 1);
  if (*ld < cols || *ld > kMaxLd)
    return fail(TG_E_LAYOUT, std::string(name) + fmt(" %lld must be 0 (packed) or %lld .. 2^40", *ld, cols));
  if (rows > kMaxSpan / *ld)
    return fail(TG_E_LAYOUT, std::string(name) + fmt(" %lld puts %lld rows past any address space", *ld, rows));
  return TG_OK;
}
bool misaligned(const void* p, int eb) { return (uintptr_t)p % (uintptr_t)eb != 0; }

int check_extents(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0)
    return fail(TG_E_SHAPE, fmt("negative extent (M=%lld, N=%lld, K=%lld)", M, N, K));
  if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return fail(TG_E_SHAPE, "extent above 2^30");
  return TG_OK;
}
int check_workspace(const void* ws, int64_t bytes) {
  if (bytes < 0) return fail(TG_E_ARG, "workspace_bytes is negative");
  if (bytes > 0 && !ws) return fail(TG_E_NULL, "workspace is NULL");
  if (misaligned(ws, 16)) return fail(TG_E_ALIGN, "workspace must be 16-byte aligned");
  return TG_OK;
}

// ------------------------------------------------------------- the product's kernel choice ----

// How a problem is cut: kernel family, block size and parts of K.  `budget`: workspace bytes
// (-1: as much as the best plan wants).
struct EpChoice {
  int kernel, bs, splits;
  int64_t kps, ws;
  int waves, cn;   // of a TOKENS workgroup
  bool ring;       // direct blocks in the four-stage ring
};

// Floats of a row of partial sums: whole 32 bytes; gated (N columns of both projections together): for each of them.
int64_t part_ld(int64_t N, bool gated) { return gated ? 2 * ((N / 2 + 7) / 8 * 8) : (N + 7) / 8 * 8; }

// N: columns of B; gated: half as many of D, and blocks and workgroups take half as many of either projection.
EpChoice choose_ep(int64_t M, int64_t N, int64_t K, int transB, int eb, bool direct, bool gated, int64_t budget) {
  EpChoice c{TG_EP_NONE, 0, 1, K, 0, 0, 0, false};
  if (M == 0 || N == 0) return c;
  if (K == 0) {
    c.kernel = TG_EP_JOIN;
    c.splits = 0;
    return c;
  }
  // Few rows: the token kernel, unless blocks can take the operands directly and are faster.  Weights
  // [K][N] come to it in 64-byte runs (1 x 4096 x 4096 bf16 12.1 us, blocks 10.8; 1 x 2048 x 2048 9.0,
  // blocks 9.3); 17 to 32 rows of 16 bits read A twice over (24 x 4096 x 4096 13.2 us, blocks 11.1;
  // 32 x 1024 x 1024 5.4, blocks 6.0; fp8 32 x 8192 x 4096 11.6, blocks 12.9).
  const bool blocks_win = direct && (!transB ? N * K > (int64_t)1 << 23 : M > 16 && eb == 2 && N * K > (int64_t)1 << 22);
  // gated weights [K][2N]: blocks alone (1 x 2·8192 x 4096 bf16 36 us, [2N][K] here 30; 32 rows 39, 31)
  if (M <= kTokenRows && !blocks_win && (transB || !gated)) {
    c.kernel = TG_EP_TOKENS;
    if (transB) {
      // a workgroup for every CU, and no more where N has them to spare
      c.cn = N >= 8192 ? 32 : N >= 4096 ? 16 : N >= 2048 ? 8 : 4;
      if (gated) c.cn = std::max(4, c.cn / 2);
    } else {
      // 64 bytes of each k-row: parts of K of at least 1024 rows (64 KB, 2.5 us, where the join costs
      // 3 us) while there are fewer than 256 workgroups
      c.cn = 32;
      const int64_t per = M * part_ld(N, gated) * 4;
      int64_t s = std::min<int64_t>(256 / ((N + 31) / 32), K / 1024);
      if (budget >= 0) s = std::min(s, budget / per);
      if (s >= 2) {
        c.kps = ((K + s - 1) / s + 31) / 32 * 32;
        c.splits = (int)((K + c.kps - 1) / c.kps);
        c.ws = per * c.splits;
      }
    }
    c.waves = (int)std::min<int64_t>(16, (c.kps * eb + 127) / 128);   // a step of K each at least
    return c;
  }
  auto blocks = [&](int64_t b) { return ((M + b - 1) / b) * ((N + b - 1) / b); };
  // Times below: bf16, MI355X, M x N x K.  Gated products and products of integers go by the same bounds, by the columns
  // of B and the bytes of K; theirs were not swept (gated bf16 of 2·8192 x 4096 weights, us: 128 rows 45, 512 rows 80,
  // 2048 rows 203).
  const int64_t bk = 128 / eb, steps = (K + bk - 1) / bk;
  c.kernel = direct ? TG_EP_DIRECT : TG_EP_STAGED;
  int64_t s = 1;   // parts of K
  if (direct && (blocks(256) >= 256 || blocks(128) > 512)) {
    // 256-wide blocks once they fill the chip (2048 x 4096 x 4096, 128 of them: 77 us, 128-wide 69)
    c.bs = 256;
  } else if (direct && blocks(256) >= 112 && blocks(256) <= 128 && steps >= 96) {
    // half the chip's worth and a long sum: two parts (4096 x 2048 x 8192: 129 us, 128-wide 138)
    c.bs = 256;
    s = 2;
  } else if (blocks(128) >= 192) {
    // 128-wide; at most one a CU: the ring of four stages (2048 x 2048 x 2048: 23.7 us, two stages
    // 28.3), else two workgroups of two stages on a CU (2048 x 3000 x 1000: 26.9 us, ring 30.8)
    c.bs = 128;
    c.ring = direct && blocks(128) <= 256;
  } else if (direct && blocks(128) <= 128 && blocks(64) * steps >= 256 * 128) {
    // 128-wide in parts where 64-wide ones would be bound by the L2, which both feed from at about
    // 13 TB/s and 64-wide ones ask twice as much of (256 x 4096 x 8192: 36 us, 64-wide 42;
    // 256 x 4096 x 4096: 22, 64-wide 18)
    c.bs = 128;
    c.ring = true;
    s = std::min(256 / blocks(128), steps / 16);
  } else {
    // 64-wide (1024 x 1024 x 1024: 7.1 us, 128-wide 11.4), and parts of K of at least 16 stages while
    // they leave CUs without work (64 x 4096 x 4096: one part 16.4 us, four 12.6, eight 13.8)
    c.bs = 64;
    c.ring = direct;
    s = std::min(256 / blocks(64), steps / 16);
  }
  const int64_t per = M * part_ld(N, gated) * 4;
  if (budget >= 0) s = std::min(s, budget / per);
  if (s < 2) return c;
  int64_t each = (steps + s - 1) / s;
  if (c.bs == 256) each += each & 1;   // whole stage pairs
  c.splits = (int)((steps + each - 1) / each);
  c.kps = each * bk;
  if (c.splits < 2) {
    c.splits = 1;
    c.kps = K;
    return c;
  }
  c.ws = per * c.splits;
  return c;
}

// Whether the direct loads can serve an operand: 16-byte chunks aligned and inside a row, and
// every 32-bit offset of a block's panel below 2^31.
bool direct_operand(const void* p, int64_t ld, bool mn, int64_t extent, int64_t K, int eb) {
  if (misaligned(p, 16) || (ld * eb) % 16) return false;
  if (mn) return (extent * eb) % 16 == 0 && (K + 512) * ld * eb < kDirectSpan;
  return (K * eb) % 16 == 0 && 256 * ld * eb + K * eb + 1024 < kDirectSpan;
}

int plan_ep(const void* A, const void* B, const void* D, int64_t M, int64_t N, int64_t K, int64_t lda,
            int64_t ldb, int64_t ldd, int transA, int transB, int a_dtype, int b_dtype, int d_dtype,
            const tg_epilogue* ep, const void* ws, int64_t ws_bytes, tg_ep_plan* plan, EpArgs* g, bool gated = false) {
  static const tg_epilogue kNone{};
  if (!ep) ep = &kNone;
  const int64_t W = gated && N <= kMaxDim ? 2 * N : N;   // columns of B
  int st = check_extents(M, W, K);
  if (st) return st;
  if (gated && ep->residual) return fail(TG_E_ARG, "a gated product takes no residual");
  if (gated && transA) return fail(TG_E_LAYOUT, "a gated product's A is stored [M,K]");
  if (!((is16(a_dtype) || a_dtype == TG_I8) && a_dtype == b_dtype) && !(isf8(a_dtype) && isf8(b_dtype)))
    return fail(TG_E_DTYPE, fmt("operands must both be TG_F16, both TG_BF16, both TG_I8, or both fp8 (got %lld, %lld)",
                                a_dtype, b_dtype));
  if (a_dtype == TG_I8 && K > kMaxIntK)
    return fail(TG_E_SHAPE, fmt("K %lld: sums of 8-bit integers are held in 32 bits, K is at most %lld", K, kMaxIntK));
  if (!is_float(d_dtype)) return fail(TG_E_DTYPE, fmt("d_dtype must be TG_F16, TG_BF16 or TG_F32 (got %lld)", d_dtype));
  if (ep->bias && !is_float(ep->bias_dtype))
    return fail(TG_E_DTYPE, fmt("bias_dtype must be TG_F16, TG_BF16 or TG_F32 (got %lld)", ep->bias_dtype));
  if (transA != 0 && transA != 1) return fail(TG_E_ARG, "transA must be 0 or 1");
  if (transB != 0 && transB != 1) return fail(TG_E_ARG, "transB must be 0 or 1");
  if (ep->act < TG_ACT_NONE || ep->act > TG_ACT_SILU) return fail(TG_E_ARG, fmt("unknown activation %lld", ep->act));
  if (is8(a_dtype) && (transA || !transB))
    return fail(TG_E_LAYOUT, "8-bit operands are stored A [M,K], B [N,K] (transA 0, transB 1)");
  int64_t ldr = ep->ld_residual, ldz = ep->ld_z;
  if ((st = resolve_ld("lda", &lda, transA ? M : K, transA ? K : M)) ||
      (st = resolve_ld("ldb", &ldb, transB ? K : W, transB ? W : K)) ||
      (st = resolve_ld("ldd", &ldd, N, M)) || (ep->residual && (st = resolve_ld("ld_residual", &ldr, N, M))) ||
      (ep->Z && (st = resolve_ld("ld_z", &ldz, W, M))))
    return st;
  if ((st = check_workspace(ws, ws_bytes))) return st;
  *plan = tg_ep_plan{};
  if (M == 0 || N == 0) return TG_OK;
  if (!D) return fail(TG_E_NULL, "D is NULL");
  if (K > 0 && (!A || !B)) return fail(TG_E_NULL, "A or B is NULL");
  const int eb = bytes_of(a_dtype), db = bytes_of(d_dtype);
  if ((K > 0 && (misaligned(A, eb) || misaligned(B, eb))) || misaligned(D, db) ||
      (ep->residual && misaligned(ep->residual, db)) || misaligned(ep->Z, db) ||
      (ep->bias && misaligned(ep->bias, bytes_of(ep->bias_dtype))) || misaligned(ep->row_scale, 4) ||
      misaligned(ep->col_scale, 4))
    return fail(TG_E_ALIGN, "a pointer is not aligned to its element");
  const Mat md = mat(D, M, N, ldd, db), mz = mat(ep->Z, M, W, ldz, db), mr = mat(ep->residual, M, N, ldr, db);
  const Mat mw = vec(ws, ws_bytes, 1);
  const Mat ins[] = {K > 0 ? mat(A, transA ? K : M, transA ? M : K, lda, eb) : Mat{},
                     K > 0 ? mat(B, transB ? W : K, transB ? K : W, ldb, eb) : Mat{},
                     ep->bias ? vec(ep->bias, W, bytes_of(ep->bias_dtype)) : Mat{}, vec(ep->row_scale, M, 4),
                     vec(ep->col_scale, W, 4)};
  for (const Mat& in : ins)
    if (overlaps(md, in) || overlaps(mz, in) || overlaps(mw, in))
      return fail(TG_E_ALIAS, "an output or the workspace overlaps an input");
  if (overlaps(mr, mz) || overlaps(mr, mw) || (overlaps(mr, md) && !same(mr, md)))
    return fail(TG_E_ALIAS, "the residual overlaps an output without being exactly D");
  if (overlaps(md, mz) || overlaps(md, mw) || overlaps(mz, mw))
    return fail(TG_E_ALIAS, "D, Z and the workspace must not overlap");

  // gated weights [K][2N]: chunks of either half stay inside it where N's do
  const bool direct = K > 0 && direct_operand(A, lda, transA, M, K, eb) && direct_operand(B, ldb, !transB, N, K, eb);
  const EpChoice c = choose_ep(M, W, K, transB, eb, direct, gated, ws_bytes);
  plan->kernel = c.kernel;
  plan->splits = c.splits;
  plan->k_per_split = (int32_t)c.kps;
  plan->workspace_bytes = c.ws;
  if (c.bs) {
    plan->block_m = plan->block_n = c.bs;
    plan->block_k = 128 / eb;
    plan->grid = ((M + c.bs - 1) / c.bs) * ((W + c.bs - 1) / c.bs) * c.splits;
  } else if (c.kernel == TG_EP_TOKENS) {
    plan->block_m = M <= 16 ? 16 : 32;
    plan->block_n = c.cn;
    plan->block_k = transB ? 128 / eb : 32;
    plan->grid = (N + c.cn - 1) / c.cn * c.splits;
  } else {
    plan->grid = (M * ((N + 7) / 8) + 255) / 256;
  }
  // a launch of blocks holds fewer than 2^32 threads
  const int64_t threads = c.kernel == TG_EP_TOKENS ? 64 * c.waves : c.bs == 64 ? 256 : 512;
  if ((c.kernel != TG_EP_JOIN && plan->grid * threads >= (int64_t)1 << 32) || M * ((N + 7) / 8) > ((int64_t)1 << 38))
    return fail(TG_E_SHAPE, fmt("too many output tiles (%lld workgroups of %lld threads)", plan->grid, threads));
  *g = EpArgs{};
  g->A = (const uint8_t*)A;
  g->B = (const uint8_t*)B;
  g->D = (uint8_t*)const_cast<void*>(D);
  g->lda = lda;
  g->ldb = ldb;
  g->ldd = ldd;
  g->M = (int32_t)M;
  g->N = (int32_t)N;
  g->K = (int32_t)K;
  if (c.bs) {
    g->tiles_m = (int32_t)((M + c.bs - 1) / c.bs);
    g->tiles_n = (int32_t)((W + c.bs - 1) / c.bs);   // gated: of bs / 2 results
  }
  g->waves = c.waves;
  g->cn = c.cn;
  g->ring = c.ring;
  g->splits = c.splits;
  g->k_per_split = (int32_t)c.kps;
  g->part = (float*)const_cast<void*>(ws);
  g->part_ld = part_ld(W, gated);
  g->bias = (const uint8_t*)ep->bias;
  g->res = (const uint8_t*)ep->residual;
  g->Z = (uint8_t*)ep->Z;
  g->rs = ep->row_scale;
  g->cs = ep->col_scale;
  g->ldr = ldr;
  g->ldz = ldz;
  g->bias_t = ep->bias_dtype;
  g->d_t = d_dtype;
  g->act = ep->act;
  g->ints = a_dtype == TG_I8;
  return TG_OK;
}

int hip_status(const char* what, hipError_t e) {
  if (e == hipSuccess) return TG_OK;
  return fail(TG_E_HIP, std::string(what) + " launch: " + hipGetErrorString(e));
}

int run_ep(const EpArgs& g, const tg_ep_plan& p, int transA, int transB, int a_dtype, int b_dtype, hipStream_t s,
           bool fine = false) {
  if (p.kernel == TG_EP_NONE) return TG_OK;
  if (p.kernel != TG_EP_JOIN) {
    const int st = hip_status("tile_gemm_ep", p.kernel == TG_EP_TOKENS
                                                  ? launch_ep_tokens(g, transA, transB, a_dtype, b_dtype, g.waves, s)
                                                  : launch_ep_block(g, transA, transB, a_dtype, b_dtype,
                                                                    {p.block_m, p.kernel == TG_EP_STAGED, g.ring != 0, fine}, s));
    if (st || g.splits == 1) return st;
  }
  return hip_status("tile_gemm_ep join", launch_ep_join(g, false, s));
}
int run_gated(const EpArgs& g, const tg_ep_plan& p, int transB, int a_dtype, int b_dtype, hipStream_t s) {
  if (p.kernel == TG_EP_NONE) return TG_OK;
  if (p.kernel != TG_EP_JOIN) {
    const int st = hip_status("tile_gemm_gated", p.kernel == TG_EP_TOKENS
                                                     ? launch_gated_tokens(g, a_dtype, b_dtype, g.waves, s)
                                                     : launch_gated_block(g, transB, a_dtype, b_dtype,
                                                                          {p.block_m, p.kernel == TG_EP_STAGED, g.ring != 0}, s));
    if (st || g.splits == 1) return st;
  }
  return hip_status("tile_gemm_gated join", launch_ep_join(g, true, s));
}

// Row groups of the bias gradient, one workgroup each per 64 columns: one up to 256 rows (no second
// launch), else about 2048 workgroups of at least 64 rows.
int64_t bias_groups(int64_t M, int64_t N) {
  if (M <= 256) return 1;
  const int64_t cols = std::max<int64_t>(1, (N + 63) / 64);
  return std::min((M + 63) / 64, std::max<int64_t>(1, (2047 + cols) / cols));
}

// Workgroups of the norm's backward pass, each with a row (four short rows) at least.  More of them
// keep more rows in flight but write and add more shares of dW: 16384 x 4096 bf16 103 us with 512
// (256: 118, 1024: 107), 8192 x 8192 104 us with 256 (512: 109).
// The layer norm's shares are twice as long: 512 only from 2048 rows on (bf16, us a call with 256 and with 512: 1003 x
// 4096 14.9, 17.4; 1500 x 2048 13.6, 13.7; 2000 x 4096 18.8, 19.2; 2048 x 2048 15.9, 14.1; 4096 x 2048 24.0, 18.9;
// 16384 x 4096 103, 82).
int64_t norm_groups(NormKind kind, int64_t rows, int64_t cols) {
  const int64_t per = cols <= 1024 && norm_in_registers(cols) ? 4 : 1;
  const int64_t most = cols <= 4096 && (kind == kRms || rows >= 2048) ? 512 : 256;
  return std::max<int64_t>(1, std::min<int64_t>((rows + per - 1) / per, most));
}

// ---------------------------------------------------------------------------- the norms ----

const char* const kNormName[] = {"tile_rmsnorm", "tile_layernorm", "tile_quantize_rows"};
const char* const kNormBwdName[] = {"tile_rmsnorm_bwd", "tile_layernorm_bwd"};

int run_norm(NormKind kind, const void* X, const void* R, const void* W, const void* B, void* H, void* Y, void* S,
             float* mean, float* rstd, int64_t rows, int64_t cols, int64_t ld_x, int64_t ld_r, int64_t ld_h,
             int64_t ld_y, float eps, int dtype, int w_dtype, int y_dtype, int scale_kind, void* stream) {
  clear_error();
  if (rows < 0 || rows > kMaxDim || cols < 1 || cols > kMaxDim)
    return fail(TG_E_SHAPE, fmt("rows must be 0 .. 2^30 and cols 1 .. 2^30 (got %lld, %lld)", rows, cols));
  if (!is_float(dtype)) return fail(TG_E_DTYPE, fmt("dtype must be TG_F16, TG_BF16 or TG_F32 (got %lld)", dtype));
  if (w_dtype != dtype && w_dtype != TG_F32) return fail(TG_E_DTYPE, "w_dtype must be dtype or TG_F32");
  if (scale_kind < TG_SCALE_NONE || scale_kind > TG_SCALE_BLOCK)
    return fail(TG_E_ARG, fmt("unknown scale kind %lld", scale_kind));
  if (kind == kRows && scale_kind == TG_SCALE_NONE) return fail(TG_E_ARG, "quantised rows need scales: TG_SCALE_ROW or TG_SCALE_BLOCK");
  if (scale_kind == TG_SCALE_NONE    ? y_dtype != dtype
      : scale_kind == TG_SCALE_BLOCK ? !isf8(y_dtype)
                                     : !is8(y_dtype))
    return fail(TG_E_DTYPE, "y_dtype must be dtype without scales, TG_FP8_E4M3 or TG_FP8_E5M2 with them, or TG_I8 with row scales");
  if (scale_kind == TG_SCALE_BLOCK && cols % 32)
    return fail(TG_E_SHAPE, fmt("block scales need cols %% 32 == 0 (got %lld)", cols));
  if (!(eps >= 0.0f) || std::isinf(eps)) return fail(TG_E_ARG, "eps must be finite and not negative");
  if (H && !R) return fail(TG_E_ARG, "H is the sum X + R: it needs R");
  int st;
  if ((st = resolve_ld("ld_x", &ld_x, cols, rows)) || (st = resolve_ld("ld_r", &ld_r, cols, rows)) ||
      (st = resolve_ld("ld_h", &ld_h, cols, rows)) || (st = resolve_ld("ld_y", &ld_y, cols, rows)))
    return st;
  if (rows == 0) return TG_OK;
  if (!X || (!W && kind != kRows) || !Y) return fail(TG_E_NULL, kind == kRows ? "X or Y is NULL" : "X, W or Y is NULL");
  if (scale_kind != TG_SCALE_NONE && !S) return fail(TG_E_NULL, "scales need S");
  const int eb = bytes_of(dtype), yb = bytes_of(y_dtype), wb = bytes_of(w_dtype);
  if (misaligned(X, eb) || misaligned(R, eb) || misaligned(H, eb) || misaligned(Y, yb) || misaligned(W, wb) ||
      misaligned(B, wb) || misaligned(mean, 4) || misaligned(rstd, 4) || (scale_kind == TG_SCALE_ROW && misaligned(S, 4)))
    return fail(TG_E_ALIGN, "a pointer is not aligned to its element");
  const Mat mx = mat(X, rows, cols, ld_x, eb), mr = mat(R, rows, cols, ld_r, eb), mh = mat(H, rows, cols, ld_h, eb);
  const Mat outs[] = {mat(Y, rows, cols, ld_y, yb), vec(rstd, rows, 4),
                      scale_kind == TG_SCALE_ROW ? vec(S, rows, 4)
                      : scale_kind == TG_SCALE_BLOCK ? vec(S, rows * (cols / 32), 1) : Mat{}, vec(mean, rows, 4)};
  const Mat mw = vec(W, cols, wb), mb = vec(B, cols, wb);
  for (int i = 0; i < 4; ++i) {
    if (overlaps(outs[i], mx) || overlaps(outs[i], mr) || overlaps(outs[i], mw) || overlaps(outs[i], mb) || overlaps(outs[i], mh))
      return fail(TG_E_ALIAS, "an output overlaps an input or H");
    for (int j = i + 1; j < 4; ++j)
      if (overlaps(outs[i], outs[j])) return fail(TG_E_ALIAS, "outputs overlap each other");
  }
  if ((overlaps(mh, mx) && !same(mh, mx)) || (overlaps(mh, mr) && !same(mh, mr)) || overlaps(mh, mw) || overlaps(mh, mb))
    return fail(TG_E_ALIAS, "H overlaps an input without being exactly X or R");
  NormArgs a{};
  a.X = (const uint8_t*)X;
  a.R = (const uint8_t*)R;
  a.W = (const uint8_t*)W;
  a.B = (const uint8_t*)B;
  a.H = (uint8_t*)H;
  a.Y = (uint8_t*)Y;
  a.S = (uint8_t*)S;
  a.rstd = rstd;
  a.mean = mean;
  a.rows = rows;
  a.cols = cols;
  a.ldx = ld_x;
  a.ldr = ld_r;
  a.ldh = ld_h;
  a.ldy = ld_y;
  a.eps = eps;
  a.w_t = w_dtype;
  a.y_t = y_dtype;
  hipStream_t s = (hipStream_t)stream;
  return hip_status(kNormName[kind], kind == kRms     ? launch_rmsnorm(a, dtype, scale_kind, s)
                                     : kind == kLayer ? launch_layernorm(a, dtype, scale_kind, s)
                                                      : launch_quantize_rows(a, dtype, scale_kind, s));
}

// Two-pass rows: bytes that hold each row's means (kLayer has two), before the shares of the weights' gradients.
int64_t norm_dots(NormKind kind, int64_t rows, int64_t cols) {
  return norm_in_registers(cols) ? 0 : rows * (kind == kLayer ? 8 : 4);
}

int64_t norm_bwd_workspace(NormKind kind, int64_t rows, int64_t cols, int dtype) {
  if (rows < 0 || rows > kMaxDim || cols < 1 || cols > kMaxDim || !is_float(dtype)) return 0;
  const int64_t g = norm_groups(kind, rows, cols);
  return (norm_dots(kind, rows, cols) + 15) / 16 * 16 + (g > 1 ? g * cols * (kind == kLayer ? 8 : 4) : 0);
}

int run_norm_bwd(NormKind kind, const void* dY, const void* H, const void* W, const float* mean, const float* rstd,
                 const void* dH, void* dX, float* dW, float* dB, int64_t rows, int64_t cols, int64_t ld_dy, int64_t ld_h,
                 int64_t ld_dh, int64_t ld_dx, int dtype, int w_dtype, void* workspace, int64_t workspace_bytes,
                 void* stream) {
  clear_error();
  if (rows < 0 || rows > kMaxDim || cols < 1 || cols > kMaxDim)
    return fail(TG_E_SHAPE, fmt("rows must be 0 .. 2^30 and cols 1 .. 2^30 (got %lld, %lld)", rows, cols));
  if (!is_float(dtype)) return fail(TG_E_DTYPE, fmt("dtype must be TG_F16, TG_BF16 or TG_F32 (got %lld)", dtype));
  if (w_dtype != dtype && w_dtype != TG_F32) return fail(TG_E_DTYPE, "w_dtype must be dtype or TG_F32");
  int st;
  if ((st = resolve_ld("ld_dy", &ld_dy, cols, rows)) || (st = resolve_ld("ld_h", &ld_h, cols, rows)) ||
      (st = resolve_ld("ld_dh", &ld_dh, cols, rows)) || (st = resolve_ld("ld_dx", &ld_dx, cols, rows)))
    return st;
  if ((st = check_workspace(workspace, workspace_bytes))) return st;
  hipStream_t s = (hipStream_t)stream;
  if (rows > 0 && (!dY || !H || !W || !rstd || !dX)) return fail(TG_E_NULL, "dY, H, W, rstd or dX is NULL");
  if (rows > 0 && kind == kLayer && !mean) return fail(TG_E_NULL, "mean is NULL");
  const int eb = bytes_of(dtype);
  if (misaligned(dY, eb) || misaligned(H, eb) || misaligned(dH, eb) || misaligned(dX, eb) ||
      misaligned(W, bytes_of(w_dtype)) || misaligned(mean, 4) || misaligned(rstd, 4) || misaligned(dW, 4) || misaligned(dB, 4))
    return fail(TG_E_ALIGN, "a pointer is not aligned to its element");
  const Mat my = mat(dY, rows, cols, ld_dy, eb), mdh = mat(dH, rows, cols, ld_dh, eb), mdx = mat(dX, rows, cols, ld_dx, eb);
  const Mat mdw = vec(dW, cols, 4), mdb = vec(dB, cols, 4), mws = vec(workspace, workspace_bytes, 1);
  const Mat ins[] = {my, mat(H, rows, cols, ld_h, eb), mdh, vec(W, cols, bytes_of(w_dtype)), vec(rstd, rows, 4), vec(mean, rows, 4)};
  for (int i = 0; i < 6; ++i) {
    if (overlaps(mdw, ins[i]) || overlaps(mdb, ins[i]) || overlaps(mws, ins[i]))
      return fail(TG_E_ALIAS, "dW, dbias or the workspace overlaps an input");
    if (overlaps(mdx, ins[i]) && !((i == 0 && same(mdx, my)) || (i == 2 && same(mdx, mdh))))
      return fail(TG_E_ALIAS, "dX overlaps an input without being exactly dY or dH");
  }
  if (overlaps(mdx, mdw) || overlaps(mdx, mdb) || overlaps(mdx, mws) || overlaps(mdw, mws) || overlaps(mdb, mws) || overlaps(mdw, mdb))
    return fail(TG_E_ALIAS, "dX, dW, dbias and the workspace must not overlap");
  const int64_t least = norm_dots(kind, rows, cols), dots = (least + 15) / 16 * 16;   // rounded up for the shares behind it
  if (workspace_bytes < least)
    return fail(TG_E_ARG, fmt("rows of %lld columns need a workspace of at least %lld bytes", cols, least));
  if (rows == 0) {   // sums of nothing
    if (dW && (st = hip_status(kNormBwdName[kind], launch_sum_rows(dW, 0, cols, dW, s)))) return st;
    return dB ? hip_status(kNormBwdName[kind], launch_sum_rows(dB, 0, cols, dB, s)) : TG_OK;
  }
  NormBwdArgs a{};
  a.dY = (const uint8_t*)dY;
  a.H = (const uint8_t*)H;
  a.W = (const uint8_t*)W;
  a.rstd = rstd;
  a.mean = mean;
  a.dH = (const uint8_t*)dH;
  a.dX = (uint8_t*)dX;
  a.rows = rows;
  a.cols = cols;
  a.ldy = ld_dy;
  a.ldh = ld_h;
  a.ldd = ld_dh;
  a.ldx = ld_dx;
  a.w_t = w_dtype;
  a.dot = dots ? (float*)workspace : nullptr;
  int64_t groups = norm_groups(kind, rows, cols);
  float* part = (float*)((uint8_t*)workspace + dots);
  a.share_ld = cols * ((dW != nullptr) + (dB != nullptr));   // a workgroup's shares, dW's first
  if (a.share_ld) groups = std::max<int64_t>(1, std::min(groups, (workspace_bytes - dots) / (4 * a.share_ld)));
  a.dw = !dW ? nullptr : groups > 1 ? part : dW;
  a.db = !dB ? nullptr : groups > 1 ? part + (dW ? cols : 0) : dB;
  hipError_t e = kind == kRms ? launch_rmsnorm_bwd(a, dtype, groups, s) : launch_layernorm_bwd(a, dtype, groups, s);
  if ((st = hip_status(kNormBwdName[kind], e)) || !a.share_ld || groups == 1) return st;
  e = dW ? launch_sum_rows(part, groups, a.share_ld, dW, s, dB, cols) : launch_sum_rows(part, groups, cols, dB, s);
  return hip_status(kNormBwdName[kind], e);
}

}  // namespace

extern "C" {

int64_t tile_gemm_ep_workspace(int64_t M, int64_t N, int64_t K, int transA, int transB, int a_dtype) {
  if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim || (!is16(a_dtype) && !is8(a_dtype))) return 0;
  (void)transA;
  // the direct and the staged kernel can differ in block size: the larger need
  const int eb = bytes_of(a_dtype);
  return std::max(choose_ep(M, N, K, transB, eb, true, false, -1).ws, choose_ep(M, N, K, transB, eb, false, false, -1).ws);
}

int tile_gemm_ep_plan(const void* A, const void* B, const void* D, int64_t M, int64_t N, int64_t K,
                      int64_t lda, int64_t ldb, int64_t ldd, int transA, int transB, int a_dtype,
                      int b_dtype, int d_dtype, const tg_epilogue* ep, const void* workspace,
                      int64_t workspace_bytes, tg_ep_plan* out) {
  clear_error();
  if (!out) return fail(TG_E_ARG, "out is NULL");
  EpArgs g;
  return plan_ep(A, B, D, M, N, K, lda, ldb, ldd, transA, transB, a_dtype, b_dtype, d_dtype, ep, workspace,
                 workspace_bytes, out, &g);
}

int tile_gemm_ep(const void* A, const void* B, void* D, int64_t M, int64_t N, int64_t K, int64_t lda,
                 int64_t ldb, int64_t ldd, int transA, int transB, int a_dtype, int b_dtype, int d_dtype,
                 const tg_epilogue* ep, void* workspace, int64_t workspace_bytes, void* stream) {
  clear_error();
  tg_ep_plan p;
  EpArgs g;
  const int st = plan_ep(A, B, D, M, N, K, lda, ldb, ldd, transA, transB, a_dtype, b_dtype, d_dtype, ep,
                         workspace, workspace_bytes, &p, &g);
  if (st) return st;
  return run_ep(g, p, transA, transB, a_dtype, b_dtype, (hipStream_t)stream);
}

int64_t tile_gemm_ep_bwd_workspace(int64_t M, int64_t N, int64_t K, int transA, int transB, int dtype) {
  if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim || !is16(dtype)) return 0;
  const int64_t groups = bias_groups(M, N);
  int64_t ws = groups > 1 ? groups * N * 4 : 0;
  ws = std::max(ws, transA ? tile_gemm_ep_workspace(K, M, N, transB, 1, dtype)
                           : tile_gemm_ep_workspace(M, K, N, 0, !transB, dtype));
  ws = std::max(ws, transB ? tile_gemm_ep_workspace(N, K, M, 1, transA, dtype)
                           : tile_gemm_ep_workspace(K, N, M, !transA, 0, dtype));
  return ws;
}

int tile_gemm_ep_bwd(const void* dY, const void* Z, const void* A, const void* B, void* dZ, void* dA,
                     void* dB, float* dbias, int64_t M, int64_t N, int64_t K, int64_t ld_dy, int64_t ld_z,
                     int64_t lda, int64_t ldb, int transA, int transB, int dtype, int act, void* workspace,
                     int64_t workspace_bytes, void* stream) {
  return tile_gemm_ep_bwd_scaled(dY, Z, A, B, nullptr, nullptr, dZ, dA, dB, dbias, M, N, K, ld_dy, ld_z, lda, ldb,
                                 transA, transB, dtype, act, workspace, workspace_bytes, stream);
}

int tile_gemm_ep_bwd_scaled(const void* dY, const void* Z, const void* A, const void* B, const float* row_scale,
                            const float* col_scale, void* dZ, void* dA, void* dB, float* dbias, int64_t M,
                            int64_t N, int64_t K, int64_t ld_dy, int64_t ld_z, int64_t lda, int64_t ldb,
                            int transA, int transB, int dtype, int act, void* workspace, int64_t workspace_bytes,
                            void* stream) {
  clear_error();
  int st = check_extents(M, N, K);
  if (st) return st;
  if (!is16(dtype)) return fail(TG_E_DTYPE, fmt("dtype must be TG_F16 or TG_BF16 (got %lld)", dtype));
  if (transA != 0 && transA != 1) return fail(TG_E_ARG, "transA must be 0 or 1");
  if (transB != 0 && transB != 1) return fail(TG_E_ARG, "transB must be 0 or 1");
  if (act < TG_ACT_NONE || act > TG_ACT_SILU) return fail(TG_E_ARG, fmt("unknown activation %lld", act));
  if ((st = resolve_ld("ld_dy", &ld_dy, N, M)) || (st = resolve_ld("ld_z", &ld_z, N, M)) ||
      (st = resolve_ld("lda", &lda, transA ? M : K, transA ? K : M)) ||
      (st = resolve_ld("ldb", &ldb, transB ? K : N, transB ? N : K)))
    return st;
  if ((st = check_workspace(workspace, workspace_bytes))) return st;
  const bool outs = M > 0 && N > 0, scaled = row_scale || col_scale;
  if (outs && !dY) return fail(TG_E_NULL, "dY is NULL");
  if (outs && act != TG_ACT_NONE && (!Z || !dZ)) return fail(TG_E_NULL, "an activation's gradient needs Z and dZ");
  if (outs && scaled && !dZ) return fail(TG_E_NULL, "a scaled product's gradient needs dZ");
  if ((dA && outs && K > 0 && !B) || (dB && outs && K > 0 && !A))
    return fail(TG_E_NULL, "dA needs B, dB needs A");
  const void* all2[] = {dY, Z, A, B, dZ, dA, dB};
  for (const void* p : all2)
    if (misaligned(p, 2)) return fail(TG_E_ALIGN, "a pointer is not aligned to its element");
  if (misaligned(dbias, 4) || misaligned(row_scale, 4) || misaligned(col_scale, 4))
    return fail(TG_E_ALIGN, "dbias, row_scale and col_scale must be 4-byte aligned");
  const Mat my = mat(dY, M, N, ld_dy, 2), mz = mat(act != TG_ACT_NONE ? Z : nullptr, M, N, ld_z, 2);
  const Mat ma = mat(dB ? A : nullptr, transA ? K : M, transA ? M : K, lda, 2);
  const Mat mb = mat(dA ? B : nullptr, transB ? N : K, transB ? K : N, ldb, 2);
  const Mat mdz = mat(dZ, M, N, N, 2), mda = mat(dA, 1, M * K, M * K, 2), mdb = mat(dB, 1, K * N, K * N, 2);
  const Mat mbias = vec(dbias, N, 4), mw = vec(workspace, workspace_bytes, 1);
  const Mat mrs = vec(row_scale, M, 4), mcs = vec(col_scale, N, 4);
  const Mat ins[] = {my, mz, ma, mb, mrs, mcs}, results[] = {mda, mdb, mbias, mw};
  for (const Mat& o : results) {
    for (const Mat& in : ins)
      if (overlaps(o, in)) return fail(TG_E_ALIAS, "an output or the workspace overlaps an input");
    if (overlaps(o, mdz)) return fail(TG_E_ALIAS, "an output or the workspace overlaps dZ");
  }
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 4; ++j)
      if (overlaps(results[i], results[j])) return fail(TG_E_ALIAS, "outputs and the workspace must not overlap");
  if ((overlaps(mdz, my) && !same(mdz, my)) || (overlaps(mdz, mz) && !same(mdz, mz)) || overlaps(mdz, ma) ||
      overlaps(mdz, mb) || overlaps(mdz, mrs) || overlaps(mdz, mcs))
    return fail(TG_E_ALIAS, "dZ overlaps an input without being exactly dY or Z");

  // both products are planned before anything is launched
  const void* G = dZ ? dZ : dY;
  const int64_t ldg = dZ ? N : ld_dy;
  tg_ep_plan pa{}, pb{};
  EpArgs ga, gb;
  // dA[M,K] = dZ·B^T, or stored [K,M]: dA^T = B·dZ^T;  dB[K,N] = A^T·dZ, or stored [N,K]: dZ^T·A
  if (dA) {
    st = transA ? plan_ep(B, G, dA, K, M, N, ldb, ldg, 0, transB, 1, dtype, dtype, dtype, nullptr, workspace,
                          workspace_bytes, &pa, &ga)
                : plan_ep(G, B, dA, M, K, N, ldg, ldb, 0, 0, !transB, dtype, dtype, dtype, nullptr, workspace,
                          workspace_bytes, &pa, &ga);
    if (st) return st;
  }
  if (dB) {
    st = transB ? plan_ep(G, A, dB, N, K, M, ldg, lda, 0, 1, transA, dtype, dtype, dtype, nullptr, workspace,
                          workspace_bytes, &pb, &gb)
                : plan_ep(A, G, dB, K, N, M, lda, ldg, 0, !transA, 0, dtype, dtype, dtype, nullptr, workspace,
                          workspace_bytes, &pb, &gb);
    if (st) return st;
  }
  hipStream_t s = (hipStream_t)stream;
  if (dbias && N > 0 && M == 0 &&   // a sum of nothing
      (st = hip_status("tile_gemm_ep_bwd", launch_sum_rows(dbias, 0, N, dbias, s))))
    return st;
  if (outs && (dZ || dbias)) {
    int64_t groups = bias_groups(M, N);
    if (dbias) groups = std::max<int64_t>(1, std::min(groups, workspace_bytes / (4 * N)));
    ActGradArgs a{};
    a.dY = (const uint8_t*)dY;
    a.Z = (const uint8_t*)Z;
    // an unchanged dZ = dY in place is not rewritten
    a.dZ = dZ == dY && act == TG_ACT_NONE && !scaled ? nullptr : (uint8_t*)dZ;
    a.rs = row_scale;
    a.cs = col_scale;
    a.ldy = ld_dy;
    a.ldz = ld_z;
    a.M = (int32_t)M;
    a.N = (int32_t)N;
    a.rows_per = (int32_t)((M + groups - 1) / groups);
    groups = (M + a.rows_per - 1) / a.rows_per;
    a.t = dtype;
    a.act = act;
    a.sums = !dbias ? nullptr : groups > 1 ? (float*)workspace : dbias;
    if ((st = hip_status("tile_gemm_ep_bwd", launch_act_grad(a, (int)groups, s)))) return st;
    if (dbias && groups > 1 &&
        (st = hip_status("tile_gemm_ep_bwd", launch_sum_rows((const float*)workspace, groups, N, dbias, s))))
      return st;
  }
  if (dA && (st = transA ? run_ep(ga, pa, transB, 1, dtype, dtype, s) : run_ep(ga, pa, 0, !transB, dtype, dtype, s)))
    return st;
  if (dB && (st = transB ? run_ep(gb, pb, 1, transA, dtype, dtype, s) : run_ep(gb, pb, !transA, 0, dtype, dtype, s)))
    return st;
  return TG_OK;
}

int64_t tile_gemm_gated_workspace(int64_t M, int64_t N, int64_t K, int transB, int a_dtype) {
  if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim / 2 || K > kMaxDim || (!is16(a_dtype) && !is8(a_dtype))) return 0;
  const int eb = bytes_of(a_dtype);
  return std::max(choose_ep(M, 2 * N, K, transB, eb, true, true, -1).ws, choose_ep(M, 2 * N, K, transB, eb, false, true, -1).ws);
}

int tile_gemm_gated_plan(const void* A, const void* B, const void* D, int64_t M, int64_t N, int64_t K, int64_t lda,
                         int64_t ldb, int64_t ldd, int transB, int a_dtype, int b_dtype, int d_dtype,
                         const tg_epilogue* ep, const void* workspace, int64_t workspace_bytes, tg_ep_plan* out) {
  clear_error();
  if (!out) return fail(TG_E_ARG, "out is NULL");
  EpArgs g;
  return plan_ep(A, B, D, M, N, K, lda, ldb, ldd, 0, transB, a_dtype, b_dtype, d_dtype, ep, workspace, workspace_bytes,
                 out, &g, true);
}

int tile_gemm_gated(const void* A, const void* B, void* D, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb,
                    int64_t ldd, int transB, int a_dtype, int b_dtype, int d_dtype, const tg_epilogue* ep,
                    void* workspace, int64_t workspace_bytes, void* stream) {
  clear_error();
  tg_ep_plan p;
  EpArgs g;
  const int st = plan_ep(A, B, D, M, N, K, lda, ldb, ldd, 0, transB, a_dtype, b_dtype, d_dtype, ep, workspace,
                         workspace_bytes, &p, &g, true);
  if (st) return st;
  return run_gated(g, p, transB, a_dtype, b_dtype, (hipStream_t)stream);
}

int64_t tile_gemm_gated_bwd_workspace(int64_t M, int64_t N, int64_t K, int transB, int dtype) {
  if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim / 2 || K > kMaxDim || !is16(dtype)) return 0;
  const int64_t groups = bias_groups(M, N), W = 2 * N;
  int64_t ws = groups > 1 ? groups * W * 4 : 0;
  ws = std::max(ws, tile_gemm_ep_workspace(M, K, W, 0, !transB, dtype));
  ws = std::max(ws, transB ? tile_gemm_ep_workspace(W, K, M, 1, 0, dtype) : tile_gemm_ep_workspace(K, W, M, 1, 0, dtype));
  return ws;
}

int tile_gemm_gated_bwd(const void* dY, const void* Z, const void* A, const void* B, const float* row_scale,
                        const float* col_scale, void* dZ, void* dA, void* dB, float* dbias, int64_t M, int64_t N,
                        int64_t K, int64_t ld_dy, int64_t ld_z, int64_t lda, int64_t ldb, int transB, int dtype, int act,
                        void* workspace, int64_t workspace_bytes, void* stream) {
  clear_error();
  const int64_t W = N <= kMaxDim ? 2 * N : N;
  int st = check_extents(M, W, K);
  if (st) return st;
  if (!is16(dtype)) return fail(TG_E_DTYPE, fmt("dtype must be TG_F16 or TG_BF16 (got %lld)", dtype));
  if (transB != 0 && transB != 1) return fail(TG_E_ARG, "transB must be 0 or 1");
  if (act < TG_ACT_NONE || act > TG_ACT_SILU) return fail(TG_E_ARG, fmt("unknown activation %lld", act));
  if ((st = resolve_ld("ld_dy", &ld_dy, N, M)) || (st = resolve_ld("ld_z", &ld_z, W, M)) ||
      (st = resolve_ld("lda", &lda, K, M)) || (st = resolve_ld("ldb", &ldb, transB ? K : W, transB ? W : K)))
    return st;
  if ((st = check_workspace(workspace, workspace_bytes))) return st;
  const bool outs = M > 0 && N > 0;
  if (outs && (!dY || !Z || !dZ)) return fail(TG_E_NULL, "dY, Z or dZ is NULL");
  if ((dA && outs && K > 0 && !B) || (dB && outs && K > 0 && !A)) return fail(TG_E_NULL, "dA needs B, dB needs A");
  const void* all2[] = {dY, Z, A, B, dZ, dA, dB};
  for (const void* p : all2)
    if (misaligned(p, 2)) return fail(TG_E_ALIGN, "a pointer is not aligned to its element");
  if (misaligned(dbias, 4) || misaligned(row_scale, 4) || misaligned(col_scale, 4))
    return fail(TG_E_ALIGN, "dbias, row_scale and col_scale must be 4-byte aligned");
  const Mat mz = mat(Z, M, W, ld_z, 2), mdz = mat(dZ, M, W, W, 2);
  const Mat ins[] = {mat(dY, M, N, ld_dy, 2), mz, mat(dB ? A : nullptr, M, K, lda, 2),
                     mat(dA ? B : nullptr, transB ? W : K, transB ? K : W, ldb, 2), vec(row_scale, M, 4), vec(col_scale, W, 4)};
  const Mat results[] = {mat(dA, 1, M * K, M * K, 2), mat(dB, 1, K * W, K * W, 2), vec(dbias, W, 4), vec(workspace, workspace_bytes, 1)};
  for (const Mat& o : results) {
    for (const Mat& in : ins)
      if (overlaps(o, in)) return fail(TG_E_ALIAS, "an output or the workspace overlaps an input");
    if (overlaps(o, mdz)) return fail(TG_E_ALIAS, "an output or the workspace overlaps dZ");
  }
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 4; ++j)
      if (overlaps(results[i], results[j])) return fail(TG_E_ALIAS, "outputs and the workspace must not overlap");
  for (int i = 0; i < 6; ++i)
    if (overlaps(mdz, ins[i]) && !(i == 1 && same(mdz, mz))) return fail(TG_E_ALIAS, "dZ overlaps an input without being exactly Z");

  // both products are planned before anything is launched: dA[M,K] = dZ·B^T; dB[K,2N] = A^T·dZ, or stored
  // [2N,K]: dZ^T·A
  tg_ep_plan pa{}, pb{};
  EpArgs ga, gb;
  if (dA && (st = plan_ep(dZ, B, dA, M, K, W, W, ldb, 0, 0, !transB, dtype, dtype, dtype, nullptr, workspace, workspace_bytes,
                          &pa, &ga)))
    return st;
  if (dB) {
    st = transB ? plan_ep(dZ, A, dB, W, K, M, W, lda, 0, 1, 0, dtype, dtype, dtype, nullptr, workspace, workspace_bytes, &pb, &gb)
                : plan_ep(A, dZ, dB, K, W, M, lda, W, 0, 1, 0, dtype, dtype, dtype, nullptr, workspace, workspace_bytes, &pb, &gb);
    if (st) return st;
  }
  hipStream_t s = (hipStream_t)stream;
  const char* what = "tile_gemm_gated_bwd";
  if (dbias && N > 0 && M == 0 && (st = hip_status(what, launch_sum_rows(dbias, 0, W, dbias, s)))) return st;   // a sum of nothing
  if (outs) {
    int64_t groups = bias_groups(M, N);
    if (dbias) groups = std::max<int64_t>(1, std::min(groups, workspace_bytes / (4 * W)));
    ActGradArgs a{};
    a.dY = (const uint8_t*)dY;
    a.Z = (const uint8_t*)Z;
    a.dZ = (uint8_t*)dZ;
    a.rs = row_scale;
    a.cs = col_scale;
    a.ldy = ld_dy;
    a.ldz = ld_z;
    a.M = (int32_t)M;
    a.N = (int32_t)N;
    a.rows_per = (int32_t)((M + groups - 1) / groups);
    groups = (M + a.rows_per - 1) / a.rows_per;
    a.t = dtype;
    a.act = act;
    a.sums = !dbias ? nullptr : groups > 1 ? (float*)workspace : dbias;
    if ((st = hip_status(what, launch_gated_grad(a, (int)groups, s)))) return st;
    if (dbias && groups > 1 && (st = hip_status(what, launch_sum_rows((const float*)workspace, groups, W, dbias, s)))) return st;
  }
  if (dA && (st = run_ep(ga, pa, 0, !transB, dtype, dtype, s, true))) return st;
  if (dB && (st = run_ep(gb, pb, 1, 0, dtype, dtype, s, true))) return st;
  return TG_OK;
}

int tile_rmsnorm(const void* X, const void* R, const void* W, void* H, void* Y, void* S, float* rstd,
                 int64_t rows, int64_t cols, int64_t ld_x, int64_t ld_r, int64_t ld_h, int64_t ld_y, float eps,
                 int dtype, int w_dtype, int y_dtype, int scale_kind, void* stream) {
  return run_norm(kRms, X, R, W, nullptr, H, Y, S, nullptr, rstd, rows, cols, ld_x, ld_r, ld_h, ld_y, eps, dtype,
                  w_dtype, y_dtype, scale_kind, stream);
}

int tile_layernorm(const void* X, const void* R, const void* W, const void* bias, void* H, void* Y, void* S,
                   float* mean, float* rstd, int64_t rows, int64_t cols, int64_t ld_x, int64_t ld_r, int64_t ld_h,
                   int64_t ld_y, float eps, int dtype, int w_dtype, int y_dtype, int scale_kind, void* stream) {
  return run_norm(kLayer, X, R, W, bias, H, Y, S, mean, rstd, rows, cols, ld_x, ld_r, ld_h, ld_y, eps, dtype, w_dtype,
                  y_dtype, scale_kind, stream);
}

int tile_quantize_rows(const void* X, void* Y, void* S, int64_t rows, int64_t cols, int64_t ld_x, int64_t ld_y,
                       int dtype, int y_dtype, int scale_kind, void* stream) {
  return run_norm(kRows, X, nullptr, nullptr, nullptr, nullptr, Y, S, nullptr, nullptr, rows, cols, ld_x, 0, 0, ld_y,
                  0.0f, dtype, dtype, y_dtype, scale_kind, stream);
}

int64_t tile_rmsnorm_bwd_workspace(int64_t rows, int64_t cols, int dtype) {
  return norm_bwd_workspace(kRms, rows, cols, dtype);
}

int tile_rmsnorm_bwd(const void* dY, const void* H, const void* W, const float* rstd, const void* dH, void* dX,
                     float* dW, int64_t rows, int64_t cols, int64_t ld_dy, int64_t ld_h, int64_t ld_dh,
                     int64_t ld_dx, int dtype, int w_dtype, void* workspace, int64_t workspace_bytes,
                     void* stream) {
  return run_norm_bwd(kRms, dY, H, W, nullptr, rstd, dH, dX, dW, nullptr, rows, cols, ld_dy, ld_h, ld_dh, ld_dx, dtype,
                      w_dtype, workspace, workspace_bytes, stream);
}

int64_t tile_layernorm_bwd_workspace(int64_t rows, int64_t cols, int dtype) {
  return norm_bwd_workspace(kLayer, rows, cols, dtype);
}

int tile_layernorm_bwd(const void* dY, const void* H, const void* W, const float* mean, const float* rstd,
                       const void* dH, void* dX, float* dW, float* dbias, int64_t rows, int64_t cols, int64_t ld_dy,
                       int64_t ld_h, int64_t ld_dh, int64_t ld_dx, int dtype, int w_dtype, void* workspace,
                       int64_t workspace_bytes, void* stream) {
  return run_norm_bwd(kLayer, dY, H, W, mean, rstd, dH, dX, dW, dbias, rows, cols, ld_dy, ld_h, ld_dh, ld_dx, dtype,
                      w_dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
