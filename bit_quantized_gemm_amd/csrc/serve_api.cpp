// Host side of the C ABIs declared in include/atom_w8a8.h and include/atom_kv4.h: argument
// validation (all of it before any HIP call), then the kernel launches on the caller's stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "host_checks.h"
#include "serve_internal.h"

namespace {

using namespace atom::check;

// ---- KV cache
bool valid_cache(const atom_kv4_cache* c) {
  const bool dim = c->dim == 64 || c->dim == 128 || c->dim == 256;
  const bool page = c->page >= 16 && c->page <= 256 && (c->page & (c->page - 1)) == 0;
  return dim && page && c->heads >= 1 && c->heads <= 1024 && c->pages >= 1 && c->pages < (int32_t)(0x80000000u / (uint32_t)c->page);
}
struct CacheRanges {
  Range r[4];
};
CacheRanges ranges(const atom_kv4_cache* c) {
  const uint64_t rows = (uint64_t)c->pages * (uint64_t)c->heads * (uint64_t)c->page;
  return CacheRanges{{range_of(c->k, rows * (uint64_t)c->dim / 2), range_of(c->k_par, rows * 4),
                      range_of(c->v, rows * (uint64_t)c->dim / 2), range_of(c->v_par, rows * 4)}};
}
bool cache_null(const atom_kv4_cache* c) { return !c || !c->k || !c->k_par || !c->v || !c->v_par; }
bool cache_aligned(const atom_kv4_cache* c) {
  return aligned16(c->k) && aligned16(c->k_par) && aligned16(c->v) && aligned16(c->v_par);
}
bool valid_attention(int32_t total_q, int32_t q_heads, int32_t heads, int32_t dim, int32_t batch, int32_t max_q,
                     int32_t max_len) {
  if (!(dim == 64 || dim == 128 || dim == 256) || heads < 1 || heads > 1024 || q_heads < heads || q_heads % heads)
    return false;
  if (!valid_rows(total_q) || q_heads > 16384 || batch < 1 || batch > (1 << 20) || max_q < 1 || max_q > ATOM_MAX_ROWS)
    return false;
  if (max_len < 1 || max_len > (1 << 30)) return false;
  const uint64_t rows = (uint64_t)max_q * (uint64_t)(q_heads / heads);   // of one sequence and kv head
  if (rows >= ((uint64_t)1 << 30)) return false;
  const atom::Kv4Plan p = atom::kv4_plan(q_heads, heads, dim, batch, max_q, max_len);
  return (uint64_t)batch * (uint64_t)heads * (uint64_t)p.row_tiles * (uint64_t)p.chunks < (uint64_t)kv4::kMaxGroups;
}

}  // namespace

extern "C" {

int64_t atom_w8a8_row_bytes(int32_t K) {
  return valid_k8(K) ? (int64_t)row_bytes8(K) : -(int64_t)ATOM_E_SHAPE;
}

int atom_quantize_w8a8(const void* X, int64_t ldx, int32_t dtype, int32_t rows, int32_t K, void* Xq, float* sx,
                       void* stream) {
  if (!X || !Xq || !sx) return ATOM_E_NULL;
  if (!valid_k8(K) || !valid_rows(rows) || !valid_dtype(dtype)) return ATOM_E_SHAPE;
  if (!valid_x(X, ldx, rows, K)) return aligned(X, 2) ? ATOM_E_SHAPE : ATOM_E_ALIGN;
  if (!aligned16(Xq) || !aligned16(sx)) return ATOM_E_ALIGN;
  const Range in[1] = {range_of(X, x_bytes(ldx, rows, K))};
  const Range out[2] = {range_of(Xq, (uint64_t)rows * row_bytes8(K)), range_of(sx, (uint64_t)rows * 4)};
  if (int s = check_overlap(in, 1, out, 2)) return s;
  return hip_status(atom::launch_quantize_w8a8(static_cast<const uint16_t*>(X), ldx, dtype == ATOM_BF16, rows, K,
                                               static_cast<int8_t*>(Xq), sx, static_cast<hipStream_t>(stream)));
}

int atom_dequantize_w8a8(const void* Xq, const float* sx, int32_t rows, int32_t K, int32_t dtype, void* X, void* stream) {
  if (!X || !Xq || !sx) return ATOM_E_NULL;
  if (!valid_k8(K) || !valid_rows(rows) || !valid_dtype(dtype)) return ATOM_E_SHAPE;
  if (!aligned16(X) || !aligned16(Xq) || !aligned16(sx)) return ATOM_E_ALIGN;
  const Range in[2] = {range_of(Xq, (uint64_t)rows * row_bytes8(K)), range_of(sx, (uint64_t)rows * 4)};
  const Range out[1] = {range_of(X, (uint64_t)rows * (uint64_t)K * 2)};
  if (int s = check_overlap(in, 2, out, 1)) return s;
  return hip_status(atom::launch_dequantize_w8a8(static_cast<const int8_t*>(Xq), sx, rows, K, dtype == ATOM_BF16,
                                                 static_cast<uint16_t*>(X), static_cast<hipStream_t>(stream)));
}

int64_t atom_gemm_w8a8_workspace_bytes(int32_t M, int32_t N, int32_t K) {
  if (!valid_gemm8(M, N, K)) return -(int64_t)ATOM_E_SHAPE;
  return atom::w8_workspace_bytes(atom::w8_plan(M, N, K));
}

int atom_gemm_w8a8(const void* Xq, const float* sx, const void* Wq, const float* sw, const void* bias, int32_t M,
                   int32_t N, int32_t K, int32_t dtype, void* Y, void* workspace, int64_t workspace_bytes,
                   void* stream) {
  if (!Xq || !sx || !Wq || !sw || !Y) return ATOM_E_NULL;
  if (!valid_gemm8(M, N, K) || !valid_dtype(dtype)) return ATOM_E_SHAPE;
  if (!aligned16(Xq) || !aligned16(sx) || !aligned16(Wq) || !aligned16(sw) || !aligned16(bias) || !aligned16(Y))
    return ATOM_E_ALIGN;
  atom::W8Plan plan = atom::w8_plan(M, N, K);
  int64_t need = atom::w8_workspace_bytes(plan);
  if (need > 0 && (!workspace || workspace_bytes < need)) {   // too little scratch: undivided
    plan.splits = 1;
    need = 0;
  }
  if (need > 0 && !aligned16(workspace)) return ATOM_E_ALIGN;
  const Range in[5] = {range_of(Xq, (uint64_t)M * row_bytes8(K)), range_of(sx, (uint64_t)M * 4),
                       range_of(Wq, (uint64_t)N * row_bytes8(K)), range_of(sw, (uint64_t)N * 4),
                       range_of(bias, bias ? (uint64_t)N * 2 : 0)};
  const Range out[2] = {range_of(Y, (uint64_t)M * N * 2), range_of(workspace, (uint64_t)need)};
  if (int s = check_overlap(in, bias ? 5 : 4, out, need > 0 ? 2 : 1)) return s;
  return hip_status(atom::launch_gemm_w8a8(static_cast<const int8_t*>(Xq), sx, static_cast<const int8_t*>(Wq), sw,
                                           static_cast<const uint16_t*>(bias), M, N, K, dtype == ATOM_BF16,
                                           static_cast<uint16_t*>(Y), need > 0 ? static_cast<int32_t*>(workspace) : nullptr,
                                           plan, static_cast<hipStream_t>(stream)));
}

int64_t atom_linear_w8a8_workspace_bytes(int32_t M, int32_t N, int32_t K) {
  if (!valid_gemm8(M, N, K)) return -(int64_t)ATOM_E_SHAPE;
  if (atom::linear_rows_fits(M, N, K)) return 0;
  return (int64_t)((uint64_t)M * row_bytes8(K) + up16((uint64_t)M * 4)) +
         atom::w8_workspace_bytes(atom::w8_plan(M, N, K));
}

int atom_linear_w8a8(const void* X, int64_t ldx, int32_t dtype, const void* Wq, const float* sw, const void* bias,
                     int32_t M, int32_t N, int32_t K, void* Y, void* workspace, int64_t workspace_bytes,
                     void* stream) {
  if (!X || !Wq || !sw || !Y) return ATOM_E_NULL;
  if (!valid_gemm8(M, N, K) || !valid_dtype(dtype)) return ATOM_E_SHAPE;
  if (!valid_x(X, ldx, M, K)) return aligned(X, 2) ? ATOM_E_SHAPE : ATOM_E_ALIGN;
  const int64_t need = atom_linear_w8a8_workspace_bytes(M, N, K);
  if (need > 0 && !workspace) return ATOM_E_NULL;
  if (workspace_bytes < need) return ATOM_E_SHAPE;
  if (!aligned16(Wq) || !aligned16(sw) || !aligned16(bias) || !aligned16(Y) || (need > 0 && !aligned16(workspace)))
    return ATOM_E_ALIGN;
  const Range in[4] = {range_of(X, x_bytes(ldx, M, K)), range_of(Wq, (uint64_t)N * row_bytes8(K)),
                       range_of(sw, (uint64_t)N * 4), range_of(bias, bias ? (uint64_t)N * 2 : 0)};
  const Range out[2] = {range_of(Y, (uint64_t)M * N * 2), range_of(workspace, (uint64_t)need)};
  if (int s = check_overlap(in, bias ? 4 : 3, out, need > 0 ? 2 : 1)) return s;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (need == 0)
    return hip_status(atom::launch_linear_rows(static_cast<const uint16_t*>(X), ldx, static_cast<const int8_t*>(Wq), sw,
                                               static_cast<const uint16_t*>(bias), M, N, K, dtype == ATOM_BF16,
                                               static_cast<uint16_t*>(Y), st));
  int8_t* xq = static_cast<int8_t*>(workspace);
  float* sx = reinterpret_cast<float*>(xq + (uint64_t)M * row_bytes8(K));
  int32_t* part = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(sx) + up16((uint64_t)M * 4));
  const hipError_t e = atom::launch_quantize_w8a8(static_cast<const uint16_t*>(X), ldx, dtype == ATOM_BF16, M, K, xq, sx, st);
  if (e != hipSuccess) return ATOM_E_HIP;
  return hip_status(atom::launch_gemm_w8a8(xq, sx, static_cast<const int8_t*>(Wq), sw,
                                           static_cast<const uint16_t*>(bias), M, N, K, dtype == ATOM_BF16,
                                           static_cast<uint16_t*>(Y), part, atom::w8_plan(M, N, K), st));
}

int atom_kv4_append(const void* K, int64_t k_stride, const void* V, int64_t v_stride, const int64_t* slots,
                    int32_t tokens, int32_t dtype, const atom_kv4_cache* cache, void* stream) {
  if (!K || !V || !slots || cache_null(cache)) return ATOM_E_NULL;
  if (!valid_cache(cache) || !valid_rows(tokens) || !valid_dtype(dtype)) return ATOM_E_SHAPE;
  const int64_t width = (int64_t)cache->heads * cache->dim;
  if (tokens > 1 && (k_stride < width || v_stride < width || k_stride > ((int64_t)1 << 40) || v_stride > ((int64_t)1 << 40)))
    return ATOM_E_SHAPE;
  if (!aligned16(K) || !aligned16(V) || !aligned(slots, 8) || !cache_aligned(cache) ||
      (tokens > 1 && (k_stride % 8 || v_stride % 8)))
    return ATOM_E_ALIGN;
  const uint64_t kb = ((uint64_t)(tokens - 1) * (uint64_t)(tokens > 1 ? k_stride : 0) + (uint64_t)width) * 2;
  const uint64_t vb = ((uint64_t)(tokens - 1) * (uint64_t)(tokens > 1 ? v_stride : 0) + (uint64_t)width) * 2;
  const Range in[3] = {range_of(K, kb), range_of(V, vb), range_of(slots, (uint64_t)tokens * 8)};
  const CacheRanges out = ranges(cache);
  if (int s = check_overlap(in, 3, out.r, 4)) return s;
  return hip_status(atom::launch_kv4_append(static_cast<const uint16_t*>(K), k_stride, static_cast<const uint16_t*>(V),
                                            v_stride, slots, tokens, dtype == ATOM_BF16, *cache,
                                            static_cast<hipStream_t>(stream)));
}

int atom_kv4_read(const atom_kv4_cache* cache, const int64_t* slots, int32_t tokens, int32_t dtype, void* K, void* V,
                  void* stream) {
  if (!K || !V || !slots || cache_null(cache)) return ATOM_E_NULL;
  if (!valid_cache(cache) || !valid_rows(tokens) || !valid_dtype(dtype)) return ATOM_E_SHAPE;
  if (!aligned16(K) || !aligned16(V) || !aligned(slots, 8) || !cache_aligned(cache)) return ATOM_E_ALIGN;
  const uint64_t bytes = (uint64_t)tokens * (uint64_t)cache->heads * (uint64_t)cache->dim * 2;
  const CacheRanges c = ranges(cache);
  const Range in[5] = {range_of(slots, (uint64_t)tokens * 8), c.r[0], c.r[1], c.r[2], c.r[3]};
  const Range out[2] = {range_of(K, bytes), range_of(V, bytes)};
  if (int s = check_overlap(in, 5, out, 2)) return s;
  return hip_status(atom::launch_kv4_read(*cache, slots, tokens, dtype == ATOM_BF16, static_cast<uint16_t*>(K),
                                          static_cast<uint16_t*>(V), static_cast<hipStream_t>(stream)));
}

int64_t atom_kv4_attention_workspace_bytes(int32_t total_q, int32_t q_heads, int32_t heads, int32_t dim,
                                           int32_t batch, int32_t max_q, int32_t max_len) {
  if (!valid_attention(total_q, q_heads, heads, dim, batch, max_q, max_len)) return -(int64_t)ATOM_E_SHAPE;
  return atom::kv4_workspace_bytes(atom::kv4_plan(q_heads, heads, dim, batch, max_q, max_len), total_q,
                                   q_heads, dim);
}

int atom_kv4_attention(const void* Q, int64_t q_stride, const atom_kv4_cache* cache, const int32_t* table,
                       int32_t width, const int32_t* lens, const int32_t* q_start, int32_t total_q, int32_t q_heads,
                       int32_t batch, int32_t max_q, int32_t max_len, float scale, int32_t dtype, void* out,
                       void* workspace, int64_t workspace_bytes, void* stream) {
  if (!Q || !table || !lens || !q_start || !out || cache_null(cache)) return ATOM_E_NULL;
  if (!valid_cache(cache) || !valid_dtype(dtype) ||
      !valid_attention(total_q, q_heads, cache->heads, cache->dim, batch, max_q, max_len))
    return ATOM_E_SHAPE;
  if (width < 1 || (uint64_t)width * (uint64_t)cache->page > ((uint64_t)1 << 30)) return ATOM_E_SHAPE;
  if (!(scale > 0.0f) || !(scale <= 3e38f)) return ATOM_E_SHAPE;
  const int64_t qw = (int64_t)q_heads * cache->dim;
  if (total_q > 1 && (q_stride < qw || q_stride > ((int64_t)1 << 40))) return ATOM_E_SHAPE;
  if (!aligned16(Q) || (total_q > 1 && q_stride % 8) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(q_start, 4) ||
      !aligned16(out) || !cache_aligned(cache))
    return ATOM_E_ALIGN;
  atom::Kv4Plan plan = atom::kv4_plan(q_heads, cache->heads, cache->dim, batch, max_q, max_len);
  int64_t need = atom::kv4_workspace_bytes(plan, total_q, q_heads, cache->dim);
  if (need > 0 && (!workspace || workspace_bytes < need)) {   // too little scratch: undivided
    plan.chunks = 1;
    plan.chunk_tokens = max_len;
    need = 0;
  }
  if (need > 0 && !aligned16(workspace)) return ATOM_E_ALIGN;
  const CacheRanges c = ranges(cache);
  const uint64_t rows = (uint64_t)total_q;
  const Range in[8] = {range_of(Q, ((rows - 1) * (uint64_t)(total_q > 1 ? q_stride : 0) + (uint64_t)qw) * 2),
                       range_of(table, (uint64_t)batch * (uint64_t)width * 4), range_of(lens, (uint64_t)batch * 4),
                       range_of(q_start, ((uint64_t)batch + 1) * 4), c.r[0], c.r[1], c.r[2], c.r[3]};
  const Range outs[2] = {range_of(out, rows * (uint64_t)qw * 2), range_of(workspace, (uint64_t)need)};
  if (int s = check_overlap(in, 8, outs, need > 0 ? 2 : 1)) return s;
  const atom::Kv4Attention a = {static_cast<const uint16_t*>(Q), q_stride, *cache, table, lens, q_start, width, total_q,
                                q_heads, batch, max_q, max_len, scale, dtype == ATOM_BF16, static_cast<uint16_t*>(out)};
  return hip_status(atom::launch_kv4_attention(a, plan, static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

}  // extern "C"
