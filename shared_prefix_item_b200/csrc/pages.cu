// Paged KV cache: forking, growing, freeing and compacting sequences.
//
// Two kernels to a call.  One CTA decides: it checks every entry before
// anything changes (a refused call changes nothing), ranks the free pages and
// writes what is to be done to the workspace.  Then a whole grid does it:
// tables and counts, a warp per sequence, and the page copies, a warp per
// (page, layer, K or V, head).  The split keeps the decision, which needs a
// prefix sum over all entries, out of the copies, which need every SM.
#include "pages.cuh"

#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <string>

// reason of the calling thread's last failed context-free call (runtime.cu)
extern thread_local std::string g_noctx_err;

namespace duolm {

int pages_fail(int code, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_noctx_err = buf;
  return code;
}

int pages_sms(int device) {
  static std::mutex mu;
  static int sms[64] = {};
  if (device < 0 || device >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (!sms[device] && cudaDeviceGetAttribute(&sms[device], cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
    sms[device] = 0;
  return sms[device];
}

int pages_view(const duolm_pages* p, PagesView* out) {
  g_noctx_err.clear();
  if (!p) return pages_fail(DUOLM_E_ARG, "null cache");
  if (!p->k || !p->v || !p->table || !p->length || !p->refs || !p->status || !p->workspace)
    return pages_fail(DUOLM_E_ARG, "null array in the cache");
  if (p->dtype != DUOLM_DTYPE_FP32 && p->dtype != DUOLM_DTYPE_BF16 && p->dtype != DUOLM_DTYPE_FP16)
    return pages_fail(DUOLM_E_ARG, "unknown dtype %d", p->dtype);
  if (p->n_layers < 1 || p->n_kv_heads < 1 || p->n_pages < 1 || p->n_seqs < 1 || p->max_pages < 1)
    return pages_fail(DUOLM_E_ARG, "a size of the cache is below 1");
  if (p->page_tokens < 8 || p->page_tokens > 256 || (p->page_tokens & (p->page_tokens - 1)))
    return pages_fail(DUOLM_E_ARG, "page_tokens %d: a power of two in 8..256 is wanted", p->page_tokens);
  const bool f32 = p->dtype == DUOLM_DTYPE_FP32;
  if (f32 ? (p->head_dim % 32 || p->head_dim < 32 || p->head_dim > 256) : (p->head_dim != 64 && p->head_dim != 128))
    return pages_fail(DUOLM_E_ARG, "head_dim %d: 64 or 128 (16-bit), a multiple of 32 up to 256 (fp32)", p->head_dim);
  if (p->n_seqs > 1 << 20) return pages_fail(DUOLM_E_CAPACITY, "more than 2^20 sequences");
  if ((int64_t)p->max_pages * p->page_tokens > INT32_MAX / 2)
    return pages_fail(DUOLM_E_CAPACITY, "sequences of 2^30 tokens and more");
  if ((int64_t)p->n_pages * p->n_kv_heads * p->page_tokens > INT32_MAX)
    return pages_fail(DUOLM_E_CAPACITY, "a layer of 2^31 cache rows and more");
  if ((reinterpret_cast<uintptr_t>(p->k) | reinterpret_cast<uintptr_t>(p->v) | reinterpret_cast<uintptr_t>(p->status) |
       reinterpret_cast<uintptr_t>(p->workspace)) & 15)
    return pages_fail(DUOLM_E_ARG, "k, v, status and workspace must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(p->table) | reinterpret_cast<uintptr_t>(p->length) |
       reinterpret_cast<uintptr_t>(p->refs)) & 3)
    return pages_fail(DUOLM_E_ARG, "table, length and refs must be 4-byte aligned");
  if (p->workspace_bytes < pages_work_bytes(p->n_pages, p->n_seqs))
    return pages_fail(DUOLM_E_CAPACITY, "workspace of %lld bytes, %lld needed", (long long)p->workspace_bytes,
                      (long long)pages_work_bytes(p->n_pages, p->n_seqs));
  int shift = 0;
  while ((1 << shift) < p->page_tokens) ++shift;
  *out = PagesView{static_cast<char*>(p->k), static_cast<char*>(p->v), p->table, p->length, p->refs,
                   reinterpret_cast<DevStatus*>(p->status), p->n_layers, p->n_kv_heads, p->head_dim, p->page_tokens,
                   shift, p->n_pages, p->n_seqs, p->max_pages, f32 ? 4 : 2};
  return 0;
}

namespace {

// ---------------------------------------------------------------------------
// resize: entry i gets the pages for length[i] tokens, gives back what lies
// behind them, and, where it grows out of a partly filled page that others
// hold too, a copy of that page.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads) resize_plan_kernel(PagesView p, PagesWork w, int n,
                                                                   const int32_t* __restrict__ seq,
                                                                   const int32_t* __restrict__ length) {
  extern __shared__ uint32_t seen[];
  __shared__ int s_scan[32];
  __shared__ uint32_t s_err;
  pdl_launch_dependents();
  for (int i = threadIdx.x; i < (p.n_seqs + 31) / 32; i += kPlanThreads) seen[i] = 0;
  if (threadIdx.x == 0) s_err = 0;
  __syncthreads();
  pdl_wait();
  if (pages_raised(p)) return;
  int64_t need_all = 0;
  int copies = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    int need = 0, cow = 0, have = 0, want = 0;
    if (i < n) {
      const int s = seq[i], len = length ? length[i] : 0;
      if ((unsigned)s >= (unsigned)p.n_seqs || !claim(seen, s)) {
        atomicOr(&s_err, ERR_BAD_SEQ);
      } else {
        const int old = p.length[s];
        if (len < 0 || len > p.max_tokens() || old < 0 || old > p.max_tokens()) {
          atomicOr(&s_err, ERR_BAD_LENGTH);
        } else {
          have = p.pages_of(old);
          want = p.pages_of(len);
          if (len > old && (old & (p.page_tokens - 1))) {
            const int tail = p.table[(int64_t)s * p.max_pages + have - 1];
            if ((unsigned)tail >= (unsigned)p.n_pages)
              atomicOr(&s_err, ERR_BAD_INDEX);
            else
              cow = p.refs[tail] > 1;
          }
          need = min(max(want - have, 0) + cow, kScanCap);
        }
      }
    }
    int all, all_cow;
    const int at = block_scan(need, s_scan, &all);
    block_scan(cow, s_scan, &all_cow);
    if (need_all + all > p.n_pages) atomicOr(&s_err, ERR_NO_PAGES);
    if (i < n) w.entry[i] = make_int4((int)(need_all + at), have, want, cow);
    need_all += all;
    copies += all_cow;
  }
  __syncthreads();
  // the lowest free pages, in order, until there are enough
  int64_t found = 0;
  for (int64_t b = 0; !s_err && found < need_all && b < p.n_pages; b += 4 * kPlanThreads) {
    const int64_t id = b + 4 * threadIdx.x;
    int free4 = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (id + j < p.n_pages && p.refs[id + j] == 0) free4 |= 1 << j;
    int all;
    int64_t at = found + block_scan(__popc(free4), s_scan, &all);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (free4 >> j & 1) {
        if (at < need_all) w.list[at] = (int)(id + j);
        ++at;
      }
    found += all;
  }
  if (found < need_all && !s_err) {
    if (threadIdx.x == 0) raise_error(p.st, ERR_NO_PAGES, 80);
    return;
  }
  if (s_err) {
    if (threadIdx.x == 0) raise_error(p.st, s_err, 81);
    return;
  }
  if (threadIdx.x == 0) w.head[0] = copies;
  if (!copies) return;
  __syncthreads();
  // the copies, in entry order
  int done = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    const int4 e = i < n ? w.entry[i] : make_int4(0, 0, 0, 0);
    int all;
    const int at = done + block_scan(e.w, s_scan, &all);
    if (e.w) {
      const int s = seq[i];
      w.copies[at] = PageCopy{p.table[(int64_t)s * p.max_pages + e.y - 1], w.list[e.x],
                              p.length[s] & (p.page_tokens - 1), 0};
    }
    done += all;
  }
}

// Rows [0, rows) of every (layer, K or V, head) of the listed pages, a warp to
// each: 16-byte words, eight in flight per lane.  HBM bound (read + write).
__device__ __forceinline__ void copy_pages(const PagesView& p, const PageCopy* __restrict__ copies, int n, int warp,
                                           int n_warps) {
  const int lane = threadIdx.x & 31;
  const int per_page = 2 * p.n_layers * p.n_kv_heads;
  const int64_t head_words = p.head_bytes() / 16, page_words = p.page_bytes() / 16, layer_words = p.layer_bytes() / 16;
  const int row_words = p.head_dim * p.elem / 16;
  for (int64_t u = warp; u < (int64_t)n * per_page; u += n_warps) {
    const int c = (int)(u / per_page), r = (int)(u % per_page);
    const int h = r % p.n_kv_heads, lv = r / p.n_kv_heads;
    const PageCopy pc = copies[c];
    char* pool = lv & 1 ? p.v : p.k;
    const int64_t base = (int64_t)(lv >> 1) * layer_words + h * head_words;
    const uint4* src = reinterpret_cast<const uint4*>(pool) + base + pc.src * page_words;
    uint4* dst = reinterpret_cast<uint4*>(pool) + base + pc.dst * page_words;
    const int words = pc.rows * row_words;
    for (int i = lane; i < words; i += 8 * 32) {
      uint4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + 32 * j < words) v[j] = __ldcg(src + i + 32 * j);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + 32 * j < words) dst[i + 32 * j] = v[j];
    }
  }
}

__global__ void __launch_bounds__(256) resize_apply_kernel(PagesView p, PagesWork w, int n,
                                                           const int32_t* __restrict__ seq,
                                                           const int32_t* __restrict__ length) {
  pdl_launch_dependents();
  pdl_wait();
  if (pages_raised(p)) return;
  const int lane = threadIdx.x & 31;
  const int warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, n_warps = (gridDim.x * blockDim.x) >> 5;
  for (int i = warp; i < n; i += n_warps) {
    const int s = seq[i];
    const int4 e = w.entry[i];
    int32_t* row = p.table + (int64_t)s * p.max_pages;
    int next = e.x;
    if (e.w) {  // the tail first: its copy is the entry's first page
      if (lane == 0) {
        const int fresh = w.list[next];
        atomicSub(&p.refs[row[e.y - 1]], 1);
        row[e.y - 1] = fresh;
        p.refs[fresh] = 1;
      }
      ++next;
    }
    for (int j = e.y + lane; j < e.z; j += 32) {
      const int fresh = w.list[next + j - e.y];
      row[j] = fresh;
      p.refs[fresh] = 1;
    }
    for (int j = e.z + lane; j < e.y; j += 32) {
      const int gone = row[j];
      if ((unsigned)gone < (unsigned)p.n_pages)
        atomicSub(&p.refs[gone], 1);
      else
        raise_error(p.st, ERR_BAD_INDEX, 82);
      row[j] = -1;
    }
    if (lane == 0) p.length[s] = length ? length[i] : 0;
  }
  copy_pages(p, w.copies, w.head[0], warp, n_warps);
}

// ---------------------------------------------------------------------------
// fork: dst starts as the first tokens[i] tokens of src, sharing its pages.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads) fork_check_kernel(PagesView p, int n, const int32_t* __restrict__ src,
                                                                  const int32_t* __restrict__ dst,
                                                                  const int32_t* __restrict__ tokens) {
  extern __shared__ uint32_t seen[];
  __shared__ uint32_t s_err;
  pdl_launch_dependents();
  for (int i = threadIdx.x; i < (p.n_seqs + 31) / 32; i += kPlanThreads) seen[i] = 0;
  if (threadIdx.x == 0) s_err = 0;
  __syncthreads();
  pdl_wait();
  if (pages_raised(p)) return;
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int d = dst[i];
    if ((unsigned)d >= (unsigned)p.n_seqs || !claim(seen, d) || p.length[d] != 0) atomicOr(&s_err, ERR_BAD_SEQ);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int s = src[i], t = tokens[i];
    if ((unsigned)s >= (unsigned)p.n_seqs || (seen[s >> 5] >> (s & 31) & 1u))
      atomicOr(&s_err, ERR_BAD_SEQ);
    else if (t < 0 || t > p.length[s] || t > p.max_tokens())
      atomicOr(&s_err, ERR_BAD_LENGTH);
  }
  __syncthreads();
  if (threadIdx.x == 0 && s_err) raise_error(p.st, s_err, 83);
}

__global__ void __launch_bounds__(256) fork_apply_kernel(PagesView p, int n, const int32_t* __restrict__ src,
                                                         const int32_t* __restrict__ dst,
                                                         const int32_t* __restrict__ tokens) {
  pdl_launch_dependents();
  pdl_wait();
  if (pages_raised(p)) return;
  const int lane = threadIdx.x & 31;
  const int warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, n_warps = (gridDim.x * blockDim.x) >> 5;
  for (int i = warp; i < n; i += n_warps) {
    const int t = tokens[i];
    const int32_t* from = p.table + (int64_t)src[i] * p.max_pages;
    int32_t* to = p.table + (int64_t)dst[i] * p.max_pages;
    for (int j = lane; j < p.pages_of(t); j += 32) {
      const int page = from[j];
      to[j] = page;
      if ((unsigned)page < (unsigned)p.n_pages)
        atomicAdd(&p.refs[page], 1);
      else
        raise_error(p.st, ERR_BAD_INDEX, 84);
    }
    if (lane == 0) p.length[dst[i]] = t;
  }
}

// ---------------------------------------------------------------------------
// compact: with n live pages, the k-th live page at n or above moves to the
// k-th free page below n.  No page is both read and written, so the moves run
// in any order, and the old copies stay as they were.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(PagesView p, PagesWork w, int32_t* live_out) {
  __shared__ int s_scan[32];
  pdl_launch_dependents();
  pdl_wait();
  if (pages_raised(p)) return;
  int mine = 0, live;
  for (int64_t id = threadIdx.x; id < p.n_pages; id += kPlanThreads) mine += p.refs[id] > 0;
  block_scan(mine, s_scan, &live);
  int holes = 0, moved = 0;
  for (int64_t b = 0; b < p.n_pages; b += kPlanThreads) {
    const int64_t id = b + threadIdx.x;
    const int r = id < p.n_pages ? p.refs[id] : 0;
    const bool hole = id < live && r <= 0, mover = id >= live && id < p.n_pages && r > 0;
    int all;
    if (b < live) {
      const int at = block_scan(hole, s_scan, &all);
      if (hole) w.copies[holes + at].dst = (int)id;
      holes += all;
    }
    if (b + kPlanThreads > live) {
      const int at = block_scan(mover, s_scan, &all);
      if (mover) {
        PageCopy& c = w.copies[moved + at];
        c.src = (int)id;
        c.rows = p.page_tokens;
        c.refs = r;
      }
      moved += all;
    }
    if (id < p.n_pages && !mover) w.map[id] = id < live && r > 0 ? (int)id : -1;
  }
  __syncthreads();
  for (int k = threadIdx.x; k < moved; k += kPlanThreads) w.map[w.copies[k].src] = w.copies[k].dst;
  if (threadIdx.x == 0) {
    w.head[0] = moved;
    w.head[1] = live;
    *live_out = live;
  }
}

__global__ void __launch_bounds__(256) compact_apply_kernel(PagesView p, PagesWork w, int32_t* table_out,
                                                            int32_t* refs_out) {
  pdl_launch_dependents();
  pdl_wait();
  if (pages_raised(p)) return;
  const int n = w.head[0], live = w.head[1];
  const int64_t thread = blockIdx.x * (int64_t)blockDim.x + threadIdx.x, threads = gridDim.x * (int64_t)blockDim.x;
  for (int64_t i = thread; i < (int64_t)p.n_seqs * p.max_pages; i += threads) {
    const int s = (int)(i / p.max_pages), j = (int)(i % p.max_pages);
    int to = -1;
    if (j < p.pages_of(p.length[s])) {
      const int from = p.table[i];
      to = (unsigned)from < (unsigned)p.n_pages ? w.map[from] : -1;
      if (to < 0) raise_error(p.st, ERR_BAD_INDEX, 85);
    }
    table_out[i] = to;
  }
  // counts: a page that stays keeps its own, a filled hole takes its page's
  // (written below, from the list, so that refs_out may be refs itself)
  for (int64_t id = thread; id < p.n_pages; id += threads) {
    if (id >= live)
      refs_out[id] = 0;
    else if (w.map[id] >= 0)
      refs_out[id] = p.refs[id];
  }
  for (int64_t k = thread; k < n; k += threads) refs_out[w.copies[k].dst] = w.copies[k].refs;
  copy_pages(p, w.copies, n, (int)(thread >> 5), (int)(threads >> 5));
}

size_t seen_bytes(const PagesView& p) { return (size_t)((p.n_seqs + 31) / 32) * 4; }

// the bitmap of the largest cache (2^20 sequences) is 128 KB
cudaError_t allow_smem(const void* kernel, size_t bytes) {
  return bytes <= 48 * 1024 - 512
             ? cudaSuccess
             : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
}

int launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? 0 : pages_fail(DUOLM_E_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

int check_entries(const PagesView& v, int n, const char* what) {
  if (n < 0) return pages_fail(DUOLM_E_ARG, "%s: n = %d", what, n);
  if (n > v.n_seqs) return pages_fail(DUOLM_E_ARG, "%s: %d entries for %d sequences (one each)", what, n, v.n_seqs);
  return 0;
}

}  // namespace
}  // namespace duolm

using namespace duolm;

extern "C" int64_t duolm_pages_workspace(int64_t n_pages, int64_t n_seqs) {
  if (n_pages < 1 || n_seqs < 1 || n_pages > INT32_MAX || n_seqs > 1 << 20) {
    g_noctx_err = "pages_workspace: a size out of range";
    return DUOLM_E_ARG;
  }
  return pages_work_bytes(n_pages, n_seqs);
}

extern "C" int duolm_pages_resize(const duolm_pages* pages, int n, const int32_t* seq, const int32_t* length,
                                  void* cuda_stream) {
  PagesView p;
  int rc = pages_view(pages, &p);
  if (rc || (rc = check_entries(p, n, "pages_resize"))) return rc;
  if (n == 0) return 0;
  if (!seq) return pages_fail(DUOLM_E_ARG, "pages_resize: null seq");
  DeviceGuard g(pages->device);
  const int sms = pages_sms(pages->device);
  if (!g.ok() || !sms) return pages_fail(DUOLM_E_CUDA, "pages_resize: device %d", pages->device);
  const PagesWork w = pages_work(pages->workspace, p.n_pages, p.n_seqs);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(resize_plan_kernel), seen_bytes(p));
  if (e == cudaSuccess)
    e = launch_ex(resize_plan_kernel, dim3(1), dim3(kPlanThreads), seen_bytes(p), s, true, p, w, n, seq, length);
  if (e == cudaSuccess)
    e = launch_ex(resize_apply_kernel, dim3(4 * sms), dim3(256), 0, s, true, p, w, n, seq, length);
  return launched(e, "pages_resize");
}

extern "C" int duolm_pages_fork(const duolm_pages* pages, int n, const int32_t* src, const int32_t* dst,
                                const int32_t* tokens, void* cuda_stream) {
  PagesView p;
  int rc = pages_view(pages, &p);
  if (rc || (rc = check_entries(p, n, "pages_fork"))) return rc;
  if (n == 0) return 0;
  if (!src || !dst || !tokens) return pages_fail(DUOLM_E_ARG, "pages_fork: null array");
  DeviceGuard g(pages->device);
  const int sms = pages_sms(pages->device);
  if (!g.ok() || !sms) return pages_fail(DUOLM_E_CUDA, "pages_fork: device %d", pages->device);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(fork_check_kernel), seen_bytes(p));
  if (e == cudaSuccess)
    e = launch_ex(fork_check_kernel, dim3(1), dim3(kPlanThreads), seen_bytes(p), s, true, p, n, src, dst, tokens);
  if (e == cudaSuccess)
    e = launch_ex(fork_apply_kernel, dim3(std::min((n + 7) / 8, 4 * sms)), dim3(256), 0, s, true, p, n, src, dst,
                  tokens);
  return launched(e, "pages_fork");
}

extern "C" int duolm_pages_compact(const duolm_pages* pages, int32_t* table_out, int32_t* refs_out, int32_t* live_out,
                                   void* cuda_stream) {
  PagesView p;
  if (const int rc = pages_view(pages, &p)) return rc;
  if (!table_out || !refs_out || !live_out) return pages_fail(DUOLM_E_ARG, "pages_compact: null output");
  DeviceGuard g(pages->device);
  const int sms = pages_sms(pages->device);
  if (!g.ok() || !sms) return pages_fail(DUOLM_E_CUDA, "pages_compact: device %d", pages->device);
  const PagesWork w = pages_work(pages->workspace, p.n_pages, p.n_seqs);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = launch_ex(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, true, p, w, live_out);
  if (e == cudaSuccess)
    e = launch_ex(compact_apply_kernel, dim3(4 * sms), dim3(256), 0, s, true, p, w, table_out, refs_out);
  return launched(e, "pages_compact");
}

extern "C" int duolm_pages_check(const duolm_pages* pages, void* cuda_stream) {
  PagesView p;
  if (const int rc = pages_view(pages, &p)) return rc;
  DeviceGuard g(pages->device);
  if (!g.ok()) return pages_fail(DUOLM_E_CUDA, "pages_check: device %d", pages->device);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  DevStatus st{};
  cudaError_t e = cudaMemcpyAsync(&st, p.st, sizeof st, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && st.flags) e = cudaMemsetAsync(p.st, 0, sizeof st, s);
  if (e != cudaSuccess) return pages_fail(DUOLM_E_CUDA, "pages_check: %s", cudaGetErrorString(e));
  if (!st.flags) return 0;
  if (st.flags & ERR_WAIT_TIMEOUT)
    return pages_fail(DUOLM_E_DEVICE, "wait-timeout (site %u)", st.where);
  if (st.flags & ERR_BAD_INDEX)
    return pages_fail(DUOLM_E_DEVICE, "a page id in a table is out of range, or its page is free (site %u)", st.where);
  if (st.flags & ERR_BAD_SEQ)
    return pages_fail(DUOLM_E_ARG, "a sequence id out of range, used twice, or not empty where a fork goes (site %u)",
                      st.where);
  if (st.flags & ERR_BAD_LENGTH)
    return pages_fail(DUOLM_E_ARG, "a length, token count, offset or position out of range (site %u)", st.where);
  if (st.flags & ERR_STALE_PLAN)
    return pages_fail(DUOLM_E_STATE, "attention on a plan from before an error: plan the batch again (site %u)", st.where);
  return pages_fail(DUOLM_E_CAPACITY, "fewer free pages than the call needed (site %u)", st.where);
}
