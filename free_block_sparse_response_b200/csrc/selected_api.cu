// extern "C" entry points of the rotary and selected-block attention operators (see
// include/sparsepr.h for the contract): argument checks, workspace layout, launches.
#include <algorithm>
#include <cmath>
#include <cstdio>

#include "../../include/sparsepr.h"
#include "common.cuh"
#include "selected.cuh"

namespace spr {
int api_fail(int code, const char* msg);  // sets the thread's last error (api.cu)
}

namespace {

using spr::SelArgs;
using spr::View;

int bad(const char* msg) { return spr::api_fail(SPARSEPR_ERR_INVALID_ARG, msg); }
int unsupported(const char* msg) { return spr::api_fail(SPARSEPR_ERR_UNSUPPORTED, msg); }
int cuda_status(cudaError_t e, const char* where) {
  if (e == cudaSuccess) return SPARSEPR_OK;
  char buf[256];
  snprintf(buf, sizeof(buf), "%s: %s", where, cudaGetErrorString(e));
  return spr::api_fail(SPARSEPR_ERR_CUDA, buf);
}

int check_view(const sparsepr_view* v, int elem, bool aligned) {
  if (v == nullptr || v->data == nullptr) return bad("null tensor");
  if (v->stride_b < 0 || v->stride_h < 0 || v->stride_n < 0) return bad("negative stride");
  if (reinterpret_cast<uintptr_t>(v->data) % elem != 0) return bad("tensor not aligned to its type");
  const int per16 = 16 / elem;
  if (aligned && ((reinterpret_cast<uintptr_t>(v->data) & 15u) != 0 || v->stride_b % per16 != 0 ||
                  v->stride_h % per16 != 0 || v->stride_n % per16 != 0))
    return bad("tensors must start on 16-byte boundaries, with strides of whole 16-byte units");
  return SPARSEPR_OK;
}

// No two rows of an output in one place.
int check_output(const sparsepr_view* v, int32_t Bt, int32_t H, int32_t N) {
  if ((Bt > 1 && v->stride_b == 0) || (H > 1 && v->stride_h == 0) || (N > 1 && v->stride_n == 0))
    return bad("an output must not repeat rows (stride 0)");
  return SPARSEPR_OK;
}

// Key rows that repeat have no box in a tensor map (repeated heads and batch elements have).
int check_keys(const sparsepr_view* v, int32_t Nk) {
  if (Nk > 1 && v->stride_n == 0) return bad("the rows of K and V must not repeat (stride_n 0)");
  return SPARSEPR_OK;
}

int check_rest(const sparsepr_selected* p) {
  if (p->out_rest == nullptr) return SPARSEPR_OK;
  if (p->dtype != SPARSEPR_BF16) return bad("out_rest goes with bf16 results");
  if ((reinterpret_cast<uintptr_t>(p->out_rest) & 15u) != 0) return bad("out_rest must start on a 16-byte boundary");
  return SPARSEPR_OK;
}

View view(const sparsepr_view* v) { return View{v->data, v->stride_b, v->stride_h, v->stride_n}; }

int check_problem(const sparsepr_selected* p) {
  if (p == nullptr) return bad("null problem");
  if (p->dtype != SPARSEPR_BF16 && p->dtype != SPARSEPR_F32) return bad("unknown dtype");
  if (p->Bt < 1 || p->Hq < 1 || p->Hkv < 1 || p->Nq < 1 || p->Nk < 1) return bad("Bt, Hq, Hkv, Nq and Nk must be >= 1");
  if (p->Hq % p->Hkv != 0) return bad("Hq must be a multiple of Hkv");
  if (p->d != 64 && p->d != 128) return unsupported("head dim: only 64 and 128 are built");
  if (p->block != 64 && p->block != 128) return unsupported("block: only 64 and 128 are built");
  if (p->top < 1) return bad("top must be >= 1");
  if (p->causal != 0 && p->causal != 1) return bad("causal must be 0 or 1");
  if (p->n_first < 0 || p->n_local < 0) return bad("n_first and n_local must be >= 0");
  if (static_cast<long long>(p->n_first) + (p->causal ? p->n_local : 0) > p->top)
    return bad("n_first + n_local must not exceed top");
  if (!p->causal && p->n_local > 0) return bad("n_local needs causal");
  if (std::isnan(p->scale)) return bad("scale is not a number");
  const long long nb = (static_cast<long long>(p->Nk) + p->block - 1) / p->block;
  if (nb > spr::kMaxBlocks) return unsupported("more than 2048 key blocks per head");
  if (p->top > 1024) return unsupported("top above 1024");
  const long long rows = static_cast<long long>(p->Bt) * p->Hq * p->Nq;
  if (rows > (1ll << 30) || static_cast<long long>(p->Bt) * p->Hkv * p->Nk > (1ll << 30))
    return unsupported("more than 2^30 query or key rows per call");
  if (static_cast<long long>(p->Bt) * p->Hkv > 65535) return unsupported("Bt*Hkv above 65535");
  if (static_cast<long long>(p->Nq) * p->top * (p->Hq / p->Hkv) > (1ll << 30))
    return unsupported("Nq * top * Hq / Hkv above 2^30");
  return SPARSEPR_OK;
}

SelArgs base_args(const sparsepr_selected* p) {
  SelArgs a{};
  a.f32 = p->dtype == SPARSEPR_F32;
  a.causal = p->causal != 0;
  a.Bt = p->Bt, a.Hq = p->Hq, a.Hk = p->Hkv, a.group = p->Hq / p->Hkv;
  a.n = p->Nq, a.nk = p->Nk, a.d = p->d;
  a.block = p->block, a.nb = spr::ceil_div(p->Nk, p->block), a.top = p->top;
  // A causal query's own block holds keys past the query: by its mean, later keys would decide about
  // it.  So it is in whatever n_local says, unless the first blocks leave no room for a score at all.
  a.n_first = p->n_first, a.n_local = p->causal && p->n_first < p->top ? std::max(p->n_local, 1) : p->n_local;
  a.q_start0 = p->Nk - p->Nq;
  a.kv_len = p->kv_len, a.q_start = p->q_start;
  a.rest = static_cast<__nv_bfloat16*>(p->out_rest);
  a.scale = p->scale > 0.f ? p->scale : 1.0f / std::sqrt(static_cast<float>(p->d));
  return a;
}

// Bytes of partial rows that one chunk of regions may take.
constexpr size_t kPartialBytes = 1ull << 30;

// Slices, chunks and scratch regions of one call (the workspace's first 256 bytes are its
// status header).
struct Plan {
  int regions, chunk;  // chunk: regions per launch
  size_t slow, mean_parts, mean_norm2, range, key_range, offs, list, inv, units, n_units, blk, part, ml, delta, seg, acc, total;
};

Plan make_plan(SelArgs& a, bool backward) {
  Plan L{};
  const long long subs = spr::ceil_div(a.n, spr::kSub);
  // the tensor-core kernels keep their partial rows in fp16
  const size_t val = a.f32 ? sizeof(float) : 2;
  const size_t row = val * a.d + sizeof(float2);
  const size_t sub_bytes = row * spr::kSub * a.top * a.group;
  // A region is cut where its partial rows pass the chunk.  A key block's gradient is then the sum of
  // its slices', which go one after the other and add to fp32 sums of the head (acc).
  const long long per = std::min<long long>(subs, std::max<long long>(1, kPartialBytes / sub_bytes));
  a.subs = static_cast<int>(per);
  a.slice = static_cast<int>(per) * spr::kSub;
  a.slices = static_cast<int>((subs + per - 1) / per);
  // one short slice: no more room than its tokens
  if (a.slices == 1) a.slice = a.n;
  L.regions = a.Bt * a.Hk * a.slices;
  const long long entries = static_cast<long long>(a.slice) * a.top, rows = entries * a.group;
  // equal chunks, so that the last one fills the SMs too
  const long long most = std::min<long long>(L.regions, std::max<long long>(1, kPartialBytes / (row * rows)));
  L.chunk = backward && a.slices > 1 ? 1 : spr::ceil_div(L.regions, spr::ceil_div(L.regions, static_cast<int>(most)));
  // The tensor-core kernels work tile by tile.  On the fp32 pipes a unit is one CTA: long units
  // load K and V seldom (and, backward, leave few sums), short ones fill the SMs when there are
  // few rows: the longest that still gives four units per SM.
  a.unit_rows = 128;
  if (a.f32) {
    const long long all = rows * L.regions;
    a.unit_rows = backward ? 2048 : 512;
    while (a.unit_rows > 64 && all / a.unit_rows < 4 * 148) a.unit_rows /= 2;
  }
  a.unit_cap = a.nb + static_cast<int>(rows / a.unit_rows);
  // sums of split blocks: per region in fp32, two per CTA on the tensor cores
  a.seg_cap = backward && a.f32 ? static_cast<int>(2 * (rows / a.unit_rows)) + 2 : 0;
  size_t off = 256;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  const size_t R = L.regions;
  L.slow = take(sizeof(int) * (static_cast<size_t>(a.Bt) * a.Hq * a.n + 1));
  const size_t means = static_cast<size_t>(a.Bt) * a.Hk * a.nb;
  L.mean_parts = take(backward ? 0 : 2 * 2 * means * a.d);
  L.mean_norm2 = take(backward ? 0 : sizeof(float) * means);
  L.range = take(a.f32 ? 0 : sizeof(float) * means);
  L.key_range = take(a.f32 || backward ? 0 : means * a.block);
  L.offs = take(sizeof(int) * R * a.nb * a.subs);
  L.list = take(sizeof(int) * R * entries);
  L.inv = take(sizeof(int) * static_cast<size_t>(a.Bt) * a.Hk * a.n * a.top);
  L.units = take(sizeof(spr::Unit) * R * a.unit_cap);
  L.n_units = take(sizeof(int) * R);
  L.blk = take(sizeof(int4) * R * a.nb);
  L.part = take(val * a.d * rows * L.chunk);
  L.ml = take(backward && a.f32 ? 0 : sizeof(float2) * rows * L.chunk);
  L.delta = take(backward ? sizeof(float) * static_cast<size_t>(a.Bt) * a.Hq * a.n : 0);
  L.seg = take(sizeof(float) * 2 * a.block * a.d *
               (!backward ? 0 : a.f32 ? static_cast<size_t>(a.seg_cap) * L.chunk : 2 * size_t{spr::kTcShares}));
  L.acc = take(backward && a.slices > 1 ? sizeof(float) * 2 * a.nk * a.d : 0);
  L.total = off;
  return L;
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

void bind(SelArgs& a, const Plan& L, void* ws) {
  a.status = at<int>(ws, 0);
  a.slow = at<int>(ws, L.slow);
  a.mean_parts = at<char>(ws, L.mean_parts);
  a.mean_norm2 = at<float>(ws, L.mean_norm2);
  a.range = at<float>(ws, L.range);
  a.key_range = at<signed char>(ws, L.key_range);
  a.offs = at<int>(ws, L.offs);
  a.list = at<int>(ws, L.list);
  a.inv = at<int>(ws, L.inv);
  a.units = at<spr::Unit>(ws, L.units);
  a.n_units = at<int>(ws, L.n_units);
  a.blk = at<int4>(ws, L.blk);
  a.part = at<float>(ws, L.part);
  a.ml = at<float2>(ws, L.ml);
  a.delta = at<float>(ws, L.delta);
  a.seg = at<float>(ws, L.seg);
}

}  // namespace

extern "C" {

int sparsepr_rotary(const sparsepr_rotary_params* p, const double* freqs, const int32_t* positions,
                    int64_t pos_stride_b, int64_t pos_stride_n, int dtype, int32_t Bt, int32_t N, int32_t d, int32_t H1,
                    const sparsepr_view* X1, const sparsepr_view* Y1, int32_t H2, const sparsepr_view* X2,
                    const sparsepr_view* Y2, sparsepr_stream_t stream) {
  if (p == nullptr || freqs == nullptr || positions == nullptr) return bad("null pointer argument");
  if (dtype != SPARSEPR_BF16 && dtype != SPARSEPR_F32) return bad("unknown dtype");
  if (Bt < 1 || N < 1 || H1 < 1 || H2 < 0) return bad("Bt, N and H1 must be >= 1, H2 >= 0");
  if (d != 64 && d != 128) return unsupported("head dim: only 64 and 128 are built");
  if (static_cast<long long>(Bt) * N * (static_cast<long long>(H1) + H2) > (1ll << 30))
    return unsupported("more than 2^30 rows per call");
  if (p->rot_dim < 2 || p->rot_dim % 2 != 0 || p->first < 0 || p->first > d - p->rot_dim)
    return bad("the rotated part must be an even number of dims inside the head");
  if (p->layout != SPARSEPR_ROTARY_HALF && p->layout != SPARSEPR_ROTARY_INTERLEAVED) return bad("unknown rotary layout");
  if (p->inverse != 0 && p->inverse != 1) return bad("inverse must be 0 or 1");
  if (p->axes < 1 || p->axes > 4) return bad("axes must be in [1, 4]");
  int pairs = 0;
  for (int i = 0; i < p->axes; ++i) {
    if (p->pairs[i] < 0 || p->pairs[i] > p->rot_dim / 2) return bad("pairs of an axis out of range");
    pairs += p->pairs[i];
  }
  if (pairs != p->rot_dim / 2) return bad("the axes' pairs must add up to rot_dim / 2");
  if (!std::isfinite(p->factor)) return bad("factor must be finite");
  if (pos_stride_b < 0 || pos_stride_n < 0) return bad("negative stride");
  const int elem = dtype == SPARSEPR_F32 ? 4 : 2;
  int rc;
  if ((rc = check_view(X1, elem, false)) || (rc = check_view(Y1, elem, false))) return rc;
  if (H2 > 0 && ((rc = check_view(X2, elem, false)) || (rc = check_view(Y2, elem, false)))) return rc;
  if ((rc = check_output(Y1, Bt, H1, N)) || (H2 > 0 && (rc = check_output(Y2, Bt, H2, N)))) return rc;
  auto same = [](const sparsepr_view* x, const sparsepr_view* y) {
    return x->data != y->data || (x->stride_b == y->stride_b && x->stride_h == y->stride_h && x->stride_n == y->stride_n);
  };
  if (!same(X1, Y1) || (H2 > 0 && !same(X2, Y2))) return bad("in place, input and output must have the same strides");
  spr::RotaryArgs a{};
  a.x[0] = view(X1), a.y[0] = view(Y1), a.h[0] = H1, a.h[1] = H2;
  if (H2 > 0) a.x[1] = view(X2), a.y[1] = view(Y2);
  a.Bt = Bt, a.n = N, a.d = d, a.first = p->first, a.rot = p->rot_dim;
  a.half = p->layout == SPARSEPR_ROTARY_HALF;
  a.f32 = dtype == SPARSEPR_F32;
  a.inverse = p->inverse != 0;
  a.axes = p->axes;
  for (int i = 0; i < p->axes; ++i) a.pairs[i] = p->pairs[i];
  a.factor = p->factor;
  a.freqs = freqs;
  a.positions = positions, a.pos_sb = pos_stride_b, a.pos_sn = pos_stride_n;
  return cuda_status(spr::launch_rotary(a, reinterpret_cast<cudaStream_t>(stream)), "rotary");
}

size_t sparsepr_selected_workspace_size(const sparsepr_selected* p, int backward) {
  if (check_problem(p) != SPARSEPR_OK) return 0;
  SelArgs a = base_args(p);
  const size_t fwd = make_plan(a, false).total;
  SelArgs c = base_args(p);
  return backward ? std::max(fwd, make_plan(c, true).total) : fwd;
}

int sparsepr_key_means(const sparsepr_selected* p, const sparsepr_view* K, const int32_t* kv_start, int32_t max_new,
                       float* means, sparsepr_stream_t stream) {
  int rc;
  if ((rc = check_problem(p)) || (rc = check_view(K, p->dtype == SPARSEPR_F32 ? 4 : 2, true))) return rc;
  if (means == nullptr) return bad("null pointer argument");
  if (kv_start != nullptr && max_new < 1) return bad("max_new must be >= 1");
  SelArgs a = base_args(p);
  a.k = view(K);
  return cuda_status(spr::launch_key_means(a, kv_start, max_new, means, reinterpret_cast<cudaStream_t>(stream)),
                     "key means");
}

int sparsepr_select_blocks(const sparsepr_selected* p, const sparsepr_view* Q, const float* means, int32_t* sel, void* ws,
                           sparsepr_stream_t stream) {
  int rc;
  if ((rc = check_problem(p)) || (rc = check_view(Q, p->dtype == SPARSEPR_F32 ? 4 : 2, true))) return rc;
  if (means == nullptr || sel == nullptr || ws == nullptr) return bad("null pointer argument");
  if ((reinterpret_cast<uintptr_t>(means) & 15u) != 0) return bad("means must start on a 16-byte boundary");
  SelArgs a = base_args(p);
  bind(a, make_plan(a, false), ws);
  a.q = view(Q), a.means = means;
  return cuda_status(spr::launch_select(a, sel, reinterpret_cast<cudaStream_t>(stream)), "select blocks");
}

int sparsepr_selected_attn(const sparsepr_selected* p, const sparsepr_view* Q, const sparsepr_view* K,
                           const sparsepr_view* V, const int32_t* sel, const sparsepr_view* O, float* lse, void* ws,
                           sparsepr_stream_t stream) {
  int rc;
  if ((rc = check_problem(p)) || (rc = check_rest(p))) return rc;
  const int elem = p->dtype == SPARSEPR_F32 ? 4 : 2;
  for (const sparsepr_view* v : {Q, K, V, O})
    if ((rc = check_view(v, elem, true))) return rc;
  if ((rc = check_keys(K, p->Nk)) || (rc = check_keys(V, p->Nk)) || (rc = check_output(O, p->Bt, p->Hq, p->Nq))) return rc;
  if (sel == nullptr || lse == nullptr || ws == nullptr) return bad("null pointer argument");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  SelArgs a = base_args(p);
  const Plan L = make_plan(a, false);
  bind(a, L, ws);
  a.q = view(Q), a.k = view(K), a.v = view(V), a.o = view(O), a.sel = sel, a.lse = lse;
  if (spr::use_decode(a)) return cuda_status(spr::launch_decode(a, st), "selected attention: few tokens");
  if (!a.f32 && (rc = cuda_status(spr::launch_ranges(a, false, st), "selected attention: ranges"))) return rc;
  if ((rc = cuda_status(spr::launch_lists(a, st), "selected attention: lists"))) return rc;
  for (int r = 0; r < L.regions; r += L.chunk)
    if ((rc = cuda_status(spr::launch_selected_forward(a, r, std::min(L.chunk, L.regions - r), st), "selected attention")))
      return rc;
  if (a.f32) return SPARSEPR_OK;
  return cuda_status(spr::launch_mend(a, false, st), "selected attention: values outside the parts' range");
}

int sparsepr_selected_attn_backward(const sparsepr_selected* p, const sparsepr_view* dO, const sparsepr_view* Q,
                                    const sparsepr_view* K, const sparsepr_view* V, const sparsepr_view* O,
                                    const float* lse, const int32_t* sel, const sparsepr_view* dQ, const sparsepr_view* dK,
                                    const sparsepr_view* dV, void* ws, sparsepr_stream_t stream) {
  int rc;
  if ((rc = check_problem(p)) || (rc = check_rest(p))) return rc;
  const int elem = p->dtype == SPARSEPR_F32 ? 4 : 2;
  for (const sparsepr_view* v : {dO, Q, K, V, O, dQ, dK, dV})
    if ((rc = check_view(v, elem, true))) return rc;
  if ((rc = check_keys(K, p->Nk)) || (rc = check_keys(V, p->Nk)) || (rc = check_output(dQ, p->Bt, p->Hq, p->Nq)) ||
      (rc = check_output(dK, p->Bt, p->Hkv, p->Nk)) || (rc = check_output(dV, p->Bt, p->Hkv, p->Nk)))
    return rc;
  if (sel == nullptr || lse == nullptr || ws == nullptr) return bad("null pointer argument");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  SelArgs a = base_args(p);
  const Plan L = make_plan(a, true);
  bind(a, L, ws);
  a.q = view(Q), a.k = view(K), a.v = view(V), a.o = view(O), a.go = view(dO);
  a.gq = view(dQ), a.gk = view(dK), a.gv = view(dV);
  a.sel = sel, a.lse = const_cast<float*>(lse);
  if ((rc = cuda_status(spr::launch_delta(a, st), "selected attention backward: row sums"))) return rc;
  if (!a.f32 && (rc = cuda_status(spr::launch_ranges(a, true, st), "selected attention backward: ranges"))) return rc;
  if ((rc = cuda_status(spr::launch_lists(a, st), "selected attention backward: lists"))) return rc;
  a.acc = a.slices > 1 ? at<float>(ws, L.acc) : nullptr;
  for (int r = 0; r < L.regions; r += L.chunk) {
    if (a.acc != nullptr && r % a.slices == 0 &&
        (rc = cuda_status(cudaMemsetAsync(a.acc, 0, sizeof(float) * 2 * a.nk * a.d, st), "selected attention backward: sums")))
      return rc;
    if ((rc = cuda_status(spr::launch_selected_backward(a, r, std::min(L.chunk, L.regions - r), st),
                          "selected attention backward")))
      return rc;
    if (a.acc != nullptr && r % a.slices == a.slices - 1 &&
        (rc = cuda_status(spr::launch_slice_sums(a, r / a.slices, st), "selected attention backward: sums")))
      return rc;
  }
  if (a.f32) return SPARSEPR_OK;
  return cuda_status(spr::launch_mend(a, true, st), "selected attention backward: values outside the parts' range");
}

}  // extern "C"
