// attn_long.cu -- attention of drafted trees whose sequences share a prefix by
// groups (attn_shared) and over selected pages (attn_sparse).
//
// Both are attn_kernel.cuh's kernel over records that a plan kernel writes:
// - shared: a record a group, the nodes of all its sequences as rows of the
//   prefix's keys (so a prefix is read once for 256 rows of a kv head, not once a
//   sequence), and a record a sequence, its nodes over its own keys.  A row that has
//   parts of both is joined from them: softmax's sums over disjoint sets of keys add
//   up once they have a common reference.
// - sparse: a record a sequence and kv head, whose keys are the pages that any of
//   its nodes names, in order, with a word a page that says which nodes do.  A page
//   is then loaded once for all of them; the scores of those that do not name it are
//   taken out by the word.
//
// What bounds them (GB300): the chain of launches for short calls.  A plan takes 4 to 5
// us, a join 4 to 5, a kernel's first item 5 to 8: one token behind 288 shared ones 19
// us (attn_tree, which has no plan, 11), 8 x 8 nodes behind 1024 31.5, over selected
// pages 35.5.  Long prefixes: full row tiles at 2.0 us a pair and key tile (64 requests
// behind 16384 tokens, 64 / 8 heads of 128: 93 us, of which the prefix is 40, the own
// keys 38).
#include "attn_few.cuh"
#include "attn_kernel.cuh"

namespace mxg {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;

// Exclusive sum (or running maximum) over the block's threads of one value each.
template <class Op>
__device__ __forceinline__ int scan_block(int x, int none, int *s_warp, Op op, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl = op(incl, y);
  }
  __syncthreads();  // (s_warp may be in use)
  if (lane == 31) s_warp[warp] = incl;
  int excl = __shfl_up_sync(kFull, incl, 1);
  if (lane == 0) excl = none;
  __syncthreads();
  int all = none;
  for (int w = 0; w < warps; ++w) {
    if (w < warp) excl = op(excl, s_warp[w]);
    all = op(all, s_warp[w]);
  }
  if (total) *total = all;
  return excl;
}
struct Max {
  __device__ int operator()(int a, int b) const { return max(a, b); }
};
struct Sum {
  __device__ int operator()(int a, int b) const { return a + b; }
};

// A record's units (PlanUnits): strips, key tiles of each.
__device__ __forceinline__ int units_of(int strips, int tiles) {
  return (int)((uint32_t)(strips * tiles) | (strips > 1 ? kStrips : 0u));
}

// ------------------------------------------------------------------ shared
constexpr int kPlanThreads = 1024;  // at most: a thread a sequence, where there are as many
constexpr int kPlanOwn = kAttnMaxSeqs / kPlanThreads;

// One block: the sequences' nodes and contexts, the groups' sequences and
// prefixes, all within their bounds, as records and their units (key tiles of row
// groups of span[0] nodes of a group, span[1] of a sequence).
constexpr float kShortWork = 30.0f;  // us of every CTA
struct SharedLists {
  PlanRec *rec;
  int *info, *units[2], span[2];
  int *ctas;       // of the two launches, that share their work
  int most;        // CTAs of a launch
  bool one;        // there is one launch, of all records
};
__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const SharedParams p, const SharedLists to) {
  __shared__ int s_a0[kAttnMaxSeqs + 1], s_len[kAttnMaxSeqs], s_warp[kPlanThreads / 32];
  __shared__ uint16_t s_g[kAttnMaxSeqs + 1];
  pdl_trigger();
  pdl_wait();
  const AttnParams &a = p.a;
  const int threads = blockDim.x;
  const int B = a.B, page = a.cache.page_size, limit = a.table_cols * page, tid = threadIdx.x, ng = p.n_groups;
  // (what is read one after another below is on its way at once)
  if (tid * 32 <= B) {
    prefetch_l1(a.cu + tid * 32);
    if (tid * 32 < B) prefetch_l1(a.ctx + tid * 32);
    if (ng > 0 && tid * 32 <= ng) prefetch_l1(p.groups + tid * 32);
    if (tid * 32 < ng) prefetch_l1(p.prefix + tid * 32);
  }
  PlanRec *rec = to.rec;
  bool bad = false;
  // offsets never fall: a thread's own ones, then what comes before them
  auto clamp_offsets = [&](const int *at, int n, int most, auto put) {
    const int per = (n + threads - 1) / threads, b0 = min(tid * per, n), b1 = min(b0 + per, n);
    int top = 0;
    for (int b = b0; b < b1; ++b) top = max(top, min(max(__ldg(at + b), 0), most));
    int running = scan_block(top, 0, s_warp, Max(), nullptr);
    for (int b = b0; b < b1; ++b) {
      const int raw = __ldg(at + b);
      running = max(running, min(max(raw, 0), most));
      bad |= raw != running;
      put(b, running);
    }
  };
  clamp_offsets(a.cu, B + 1, a.T, [&](int b, int x) { s_a0[b] = x; });
  if (ng > 0) clamp_offsets(p.groups, ng + 1, B, [&](int g, int x) { s_g[g] = (uint16_t)x; });
  for (int g = tid; g < ng; g += threads) s_len[g] = limit;
  __syncthreads();
  // a sequence's group, or -1: the last group that begins at or before it and is not empty
  auto group_of = [&](int b) {
    if (ng == 0 || b < s_g[0] || b >= s_g[ng]) return -1;
    int lo = 0, hi = ng - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_g[mid] <= b) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  };
  int ctx[kPlanOwn], of[kPlanOwn];
#pragma unroll
  for (int i = 0; i < kPlanOwn; ++i) {
    const int b = tid + i * threads;
    of[i] = -1;
    if (b >= B) continue;
    const int raw = __ldg(a.ctx + b);
    ctx[i] = min(max(raw, 0), limit);
    bad |= raw != ctx[i] || s_a0[b + 1] - s_a0[b] > kAttnMaxNodes;
    of[i] = group_of(b);
    if (of[i] >= 0) atomicMin(&s_len[of[i]], ctx[i]);
  }
  __syncthreads();
  float work[2] = {0.0f, 0.0f};  // us of one CTA, see below
  for (int g = tid; g < ng; g += threads) {
    const int g0 = s_g[g], g1 = s_g[g + 1], raw = __ldg(p.prefix + g);
    const int len = g1 > g0 ? min(max(raw, 0), s_len[g]) & -page : 0;  // (page: a power of two)
    bad |= g1 > g0 && raw != len;
    s_len[g] = len;
    PlanRec r = {};
    r.a0 = s_a0[g0];
    r.n = s_a0[g1] - r.a0;
    r.ctx = len;
    r.hk = -1;
    r.list = (long long)g0 * a.ld_table;
    r.flags = kJoined;
    rec[g] = r;
    const int strips = div_small(r.n + to.span[0] - 1, to.span[0]) * a.Hkv, tiles = (len + kKeys - 1) / kKeys;
    to.units[0][g] = units_of(strips, tiles);
    work[0] += len > 0 ? (float)strips * (2.0f * (float)tiles + 5.0f) : 0.0f;
  }
  if (!to.one)
    for (int g = ng + tid; g < 32 * units_per_lane(ng); g += threads) to.units[0][g] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPlanOwn; ++i) {
    const int b = tid + i * threads;
    if (b >= B) continue;
    const int len = of[i] >= 0 ? s_len[of[i]] : 0, a0 = s_a0[b], a1 = s_a0[b + 1];
    PlanRec r = {};
    r.a0 = a0;
    r.n = min(a1 - a0, kAttnMaxNodes);
    r.ctx = ctx[i] - len;
    r.hk = -1;
    r.list = (long long)b * a.ld_table + (len >> (31 - __clz(page)));
    r.flags = kHasNodes | (len > 0 ? kJoined : 0);
    rec[ng + b] = r;
    const int strips = div_small(r.n + to.span[1] - 1, to.span[1]) * a.Hkv, tiles = (r.ctx + kKeys - 1) / kKeys + 1;
    to.units[1][b] = units_of(strips, tiles);
    work[1] += (float)strips * (float)(tiles + 3);
    for (int x = a0; x < a1; ++x) to.info[x] = x - a0 < kAttnMaxNodes ? len > 0 : -1;
  }
  const int before = to.one ? ng : 0;  // records of the list before the sequences'
  for (int b = B + tid; b < 32 * units_per_lane(before + B) - before; b += threads) to.units[1][b] = 0;
  for (int x = tid; x < s_a0[0]; x += threads) to.info[x] = -1;
  for (int x = s_a0[B] + tid; x < a.T; x += threads) to.info[x] = -1;
  // Two launches: estimated times, us of one CTA, are 2.0 for a prefix's key tile and 5
  // for its row group, 1.0 and 3 for a sequence's.  Where both launches are short, they
  // share the SMs and run beside one another (8 requests of 1 node behind 1024 tokens, as
  // two launches, 27 us, 32 one after the other); else each has all of them, since the
  // keys of the one held up the other's (64 requests behind 16384 tokens 105 us, 95 one
  // after the other).
  if (ng > 0 && !to.one) {
    float *const s_work = reinterpret_cast<float *>(s_len);  // (read for the last time before the barrier)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) work[i] += __shfl_xor_sync(kFull, work[i], o);
    __syncthreads();
    if ((tid & 31) == 0) s_work[tid >> 5] = work[0], s_work[32 + (tid >> 5)] = work[1];
    __syncthreads();
    if (tid == 0) {
      work[0] = work[1] = 0.0f;
      for (int w = 0; w < threads / 32; ++w) work[0] += s_work[w], work[1] += s_work[32 + w];
      const int first = (int)((float)to.most * work[0] / (work[0] + work[1]) + 0.5f);
      const int x = max(min(first, to.most - 1), 1);
      const bool both = work[0] + work[1] < kShortWork * (float)to.most;
      to.ctas[0] = both ? x : to.most;
      to.ctas[1] = both ? max(to.most - x, 1) : to.most;
    }
  } else if (tid == 0) {
    to.ctas[0] = to.ctas[1] = to.most;
  }
  if (bad && a.status) atomicOr(a.status, kBadIndex);
}

// ------------------------------------------------------------------ sparse
constexpr int kListThreads = 128;

// A block a sequence and kv head: the pages that any of its nodes names, in
// order (a bit a logical page in shared memory, a page's place is the number of bits
// below its own), and for several nodes the word of those that name it.
struct SparseLists {
  PlanRec *rec;
  int *list, *units, span;
  unsigned long long *names;
};
__global__ void __launch_bounds__(kListThreads) sparse_plan_kernel(const SparseParams p, const SparseLists to) {
  extern __shared__ uint32_t s_bits[];  // words of bits, then the number of bits before each
  __shared__ int s_warp[kListThreads / 32];
  pdl_trigger();
  const AttnParams &a = p.a;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, page = a.cache.page_size;
  int *list = to.list;
  unsigned long long *names = to.names;
  pdl_wait();
  const int *table = a.table + (long long)b * a.ld_table;
  if (tid * 32 < a.table_cols) prefetch_l1(table + tid * 32);  // (read at the end)
  const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1), raw = __ldg(a.ctx + b);
  int top = 0;
  for (int i = tid; i <= b; i += kListThreads) top = max(top, min(max(__ldg(a.cu + i), 0), a.T));
  int a0;
  scan_block(top, 0, s_warp, Max(), &a0);
  const int a1 = max(min(max(c1, 0), a.T), a0);
  const int n = min(a1 - a0, kAttnMaxNodes), ctx = min(max(raw, 0), a.table_cols * page);
  bool bad = h == 0 && (c0 != a0 || c1 != a1 || a1 - a0 > kAttnMaxNodes || raw != ctx);
  const int P = (ctx + page - 1) / page, W = (P + 31) / 32, total = n * p.n_sel;
  uint32_t *s_before = s_bits + W;
  for (int i = tid; i < W; i += kListThreads) s_bits[i] = 0;
  __syncthreads();
  // (a node's pages of this kv head follow one another, the next node's are Hkv lists on)
  const int *sel = p.sel + ((long long)a0 * a.Hkv + h) * p.n_sel;
  auto named = [&](int e, int &node) {
    node = e / p.n_sel;
    return __ldg(sel + (long long)node * a.Hkv * p.n_sel + (e - node * p.n_sel));
  };
  for (int e = tid; e < total; e += kListThreads) {
    int node;
    const int j = named(e, node);
    bad |= j >= P;
    if (j >= 0 && j < P) atomicOr(&s_bits[j >> 5], 1u << (j & 31));
  }
  __syncthreads();
  const int per = (W + kListThreads - 1) / kListThreads, w0 = min(tid * per, W), w1 = min(w0 + per, W);
  int sum = 0, count;
  for (int i = w0; i < w1; ++i) sum += __popc(s_bits[i]);
  int at = scan_block(sum, 0, s_warp, Sum(), &count);
  const long long base = ((long long)a0 * a.Hkv + (long long)h * n) * p.n_sel;
  for (int i = w0; i < w1; ++i) {
    s_before[i] = at;
    at += __popc(s_bits[i]);
  }
  if (n > 1)
    for (int i = tid; i < count; i += kListThreads) names[base + i] = 0;
  __syncthreads();
  // (several nodes name a page: they write the same number)
  for (int e = tid; e < total; e += kListThreads) {
    int node;
    const int j = named(e, node);
    if (j >= 0 && j < P) {
      const long long x = base + s_before[j >> 5] + __popc(s_bits[j >> 5] & ((1u << (j & 31)) - 1u));
      list[x] = __ldg(table + j);
      if (n > 1) atomicOr(names + x, 1ull << node);
    }
  }
  if (tid == 0) {
    const bool has_last = P > 0 && (s_bits[(P - 1) >> 5] >> ((P - 1) & 31) & 1u);
    PlanRec r = {};
    r.a0 = a0;
    r.n = n;
    r.ctx = count == 0 ? 0 : (count - 1) * page + (has_last ? ctx - (P - 1) * page : page);
    r.hk = h;
    r.list = base;
    r.flags = kHasNodes | (n > 1 ? kLists : 0);
    to.rec[b * a.Hkv + h] = r;
    to.units[b * a.Hkv + h] = units_of((n + to.span - 1) / to.span, (r.ctx + kKeys - 1) / kKeys + 1);
  }
  if (b == (int)gridDim.y - 1 && h == (int)gridDim.x - 1) {
    const int V = a.B * a.Hkv;
    for (int i = V + tid; i < 32 * units_per_lane(V); i += kListThreads) to.units[i] = 0;
  }
  if (bad && a.status) atomicOr(a.status, kBadIndex);
}

// -------------------------------------------------------------- workspaces
size_t round256(size_t n) { return (n + 255) / 256 * 256; }
size_t slots_bytes(int D, int sm_count) {
  const long long f = D == 64 ? Cfg<64, kShared>::kSlotFloats : Cfg<128, kShared>::kSlotFloats;
  return (size_t)(2 * f * (sm_count < kMaxCtas ? sm_count : kMaxCtas)) * sizeof(float);
}

// Byte offsets; a launch's items, which the join reads, come first, then its slots.
struct SharedWs {
  size_t slots, second, rec, units, ctas, info, rows, stats, end;
  SharedWs(long long N, int Hq, int D, int sm_count) {
    slots = kJoinFloats * sizeof(float);
    second = slots + slots_bytes(D, sm_count);
    rec = 2 * second;
    units = rec + 2 * kAttnMaxSeqs * sizeof(PlanRec);
    ctas = units + 2 * (kAttnMaxSeqs + 128) * sizeof(int);
    info = ctas + 16;
    rows = round256(info + N * sizeof(int));
    stats = rows + (size_t)(2 * N * Hq) * D * sizeof(float);
    end = round256(stats + (size_t)(2 * N * Hq) * 2 * sizeof(float));
  }
};
struct SparseWs {
  size_t slots, rec, units, names, list, end;
  SparseWs(long long N, int Hkv, int n_sel, int D, int sm_count) {
    slots = kJoinFloats * sizeof(float);
    rec = slots + slots_bytes(D, sm_count);
    units = rec + (size_t)kAttnMaxSeqs * Hkv * sizeof(PlanRec);
    names = units + ((size_t)kAttnMaxSeqs * Hkv + 128) * sizeof(int);
    list = names + (size_t)(N * Hkv) * n_sel * sizeof(unsigned long long);
    end = round256(list + (size_t)(N * Hkv) * n_sel * sizeof(int));
  }
};

// Sequences' rows of a kv head: where an average sequence's fit, the kernel of few
// rows (16, 32 or, sparse, 64 of them), else the one of full tiles (0).  8 requests over 16
// pages of 64, 8 heads a kv head: 1 node each 18.3 us, by full tiles 22.9; 4 nodes
// 24.9 and 31.0; 8 nodes 34.7 and 37.7.
// Shared: where sequences' strips are no more than the CTAs, full tiles too, since
// prefixes are then in the same launch (8 requests of 1 node behind 1024 tokens 23.1 us,
// by two launches 27.2; 16 25.5 and 32.3; but 32, 256 strips, behind 16384 76 and 66).
template <int MODE>
int few_rows(const AttnParams &p, int sm_count) {
  if (MODE == kShared && p.B * p.Hkv <= paged_ctas(sm_count)) return 0;
  const long long rows = ((long long)p.T + p.B - 1) / p.B * (p.Hq / p.Hkv);
  return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 && MODE == kSparse ? 64 : 0;
}
// Nodes of a row group, as the kernels cut them: those of few rows' tile, or two row tiles
// of whole nodes (12 heads a kv head: 2 * 10 nodes, not 256 / 12 = 21).
int span_of(const AttnParams &p, int rows) {
  const int G = p.Hq / p.Hkv;
  return rows ? rows / G : 2 * (kRowsT / G);
}

template <int D, int MODE>
cudaError_t launch_rows(const AttnParams &p, int sm_count, cudaStream_t stream) {
  switch (few_rows<MODE>(p, sm_count)) {
    case 16: return launch_few<D, 16, MODE>(p, sm_count, stream);
    case 32: return launch_few<D, 32, MODE>(p, sm_count, stream);
    case 64:
      if constexpr (MODE == kSparse) return launch_few<D, 64, MODE>(p, sm_count, stream);
  }
  return launch_t<D, MODE>(p, sm_count, stream);
}

// Prefixes by full tiles, and sequences beside or after them by the kernel of few rows
// -- or all of it by full tiles in one launch.
template <int D>
cudaError_t launch_shared(const SharedParams &p, AttnParams a, const SharedLists &to, int sm_count, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (to.one) {
    a.ws = a.plan.part_ws[1];
    a.plan.rec = to.rec;
    a.plan.units = to.units[0];
    a.plan.ctas = to.ctas;
    a.plan.n = p.n_groups + a.B;
    if ((e = launch_t<D, kShared>(a, sm_count, stream)) != cudaSuccess) return e;
    return launch_join<D, kShared>(a, sm_count, stream);
  }
  if (p.n_groups > 0) {
    a.ws = a.plan.part_ws[0];
    a.plan.rec = to.rec;
    a.plan.units = to.units[0];
    a.plan.ctas = to.ctas;
    a.plan.n = p.n_groups;
    if ((e = launch_t<D, kShared>(a, sm_count, stream)) != cudaSuccess) return e;
  }
  a.ws = a.plan.part_ws[1];
  a.plan.rec = to.rec + p.n_groups;
  a.plan.units = to.units[1];
  a.plan.n = a.B;
  a.plan.ctas = to.ctas + 1;
  a.plan.beside = p.n_groups > 0;
  if ((e = launch_rows<D, kShared>(a, sm_count, stream)) != cudaSuccess) return e;
  return launch_join<D, kShared>(a, sm_count, stream);
}

template <int D>
cudaError_t launch_sparse(const AttnParams &a, int sm_count, cudaStream_t stream) {
  const cudaError_t e = launch_rows<D, kSparse>(a, sm_count, stream);
  return e == cudaSuccess ? launch_join<D, kSparse>(a, sm_count, stream) : e;
}

}  // namespace

size_t attn_shared_ws_bytes(long long N, int Hq, int D, int sm_count) { return SharedWs(N, Hq, D, sm_count).end; }
size_t attn_sparse_ws_bytes(long long N, int Hkv, int n_sel, int D, int sm_count) {
  return SparseWs(N, Hkv, n_sel, D, sm_count).end;
}

cudaError_t launch_attn_shared(const SharedParams &p, int sm_count, cudaStream_t stream) {
  AttnParams a = p.a;
  const SharedWs ws(a.T, a.Hq, a.D, sm_count);
  char *w = reinterpret_cast<char *>(a.ws);
  SharedLists to = {};
  to.rec = reinterpret_cast<PlanRec *>(w + ws.rec);
  to.info = reinterpret_cast<int *>(w + ws.info);
  to.units[0] = reinterpret_cast<int *>(w + ws.units);
  const int few = few_rows<kShared>(a, sm_count);
  to.one = few == 0;
  to.units[1] = to.units[0] + (to.one ? p.n_groups : kAttnMaxSeqs + 128);
  to.ctas = reinterpret_cast<int *>(w + ws.ctas);
  to.most = paged_ctas(sm_count);
  to.span[0] = span_of(a, 0);
  to.span[1] = span_of(a, few);
  const int threads = a.B < 128 ? 128 : a.B < kPlanThreads ? (a.B + 31) / 32 * 32 : kPlanThreads;
  cudaLaunchConfig_t cfg = pdl_config(dim3(1), dim3((unsigned)threads), 0, stream);
  cudaLaunchAttribute attr[1];
  attach_pdl(cfg, attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, shared_plan_kernel, p, to);
  if (e != cudaSuccess) return e;
  a.slots = kJoinFloats;
  a.plan.info = to.info;
  a.plan.rows = reinterpret_cast<float *>(w + ws.rows);
  a.plan.stats = reinterpret_cast<float *>(w + ws.stats);
  a.plan.part_ws[1] = reinterpret_cast<float *>(w + ws.second);
  a.plan.part_ws[0] = to.one ? a.plan.part_ws[1] : p.n_groups > 0 ? reinterpret_cast<float *>(w) : nullptr;
  return a.D == 64 ? launch_shared<64>(p, a, to, sm_count, stream) : launch_shared<128>(p, a, to, sm_count, stream);
}

cudaError_t launch_attn_sparse(const SparseParams &p, int sm_count, cudaStream_t stream) {
  AttnParams a = p.a;
  const SparseWs ws(a.T, a.Hkv, p.n_sel, a.D, sm_count);
  char *w = reinterpret_cast<char *>(a.ws);
  SparseLists to = {};
  to.rec = reinterpret_cast<PlanRec *>(w + ws.rec);
  to.list = reinterpret_cast<int *>(w + ws.list);
  to.units = reinterpret_cast<int *>(w + ws.units);
  to.names = reinterpret_cast<unsigned long long *>(w + ws.names);
  to.span = span_of(a, few_rows<kSparse>(a, sm_count));
  static DeviceOnce once;
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!once.done(dev)) {
    e = cudaFuncSetAttribute(sparse_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAttnMaxListed / 32 * 8);
    if (e != cudaSuccess) return e;
    once.set(dev);
  }
  const size_t smem = (size_t)((a.table_cols + 31) / 32) * 2 * sizeof(uint32_t);
  cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)a.Hkv, (unsigned)a.B), dim3(kListThreads), smem, stream);
  cudaLaunchAttribute attr[1];
  attach_pdl(cfg, attr);
  e = cudaLaunchKernelEx(&cfg, sparse_plan_kernel, p, to);
  if (e != cudaSuccess) return e;
  a.slots = kJoinFloats;
  a.plan.rec = to.rec;
  a.plan.units = to.units;
  a.plan.n = a.B * a.Hkv;
  a.plan.list = to.list;
  a.plan.names = to.names;
  return a.D == 64 ? launch_sparse<64>(a, sm_count, stream) : launch_sparse<128>(a, sm_count, stream);
}

}  // namespace mxg
