// Attention of a chunk of query rows over a paged KV cache: the fp32 path, on
// CUDA cores (the tensor cores have no fp32 operands).
//
// One pass over the keys with a running maximum and sum: for a tile of 64
// keys, s = q.k scale (base 2), m' = max(m, max s), p = 2^(s - m'),
// l' = l 2^(m - m') + sum p, O' = O 2^(m - m') + p V; out = O / l,
// lse = ln 2 (m + log2 l).  Every statistic and O are fp32.
//
// An item's rows are (token, query head) slots of one KV head, so a K/V tile
// is read once for all heads that share it; 256 threads hold a slots x 64
// tile of scores (rows x 4 keys each) and slots x head_dim of O.
#include "pages.cuh"

namespace duolm {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;

}  // namespace

// M: slots of an item; NC: head_dim / 16, rounded up to what is instantiated
template <int M, int NC>
__global__ void __launch_bounds__(kThreads) attention_simt_kernel(PagesView p, PagesPlan pl, AttnArgs a) {
  constexpr int RM = M / 16;
  constexpr int E = 4;
  extern __shared__ float smem[];
  __shared__ int s_last;
  const int hd = p.head_dim, ld = hd + 4, nc = hd / 16, words = hd / E;
  float* Qs = smem;
  float* Ks = Qs + M * ld;
  float* Vs = Ks + kTile * ld;
  float* Ps = Vs + kTile * hd;
  pdl_launch_dependents();
  pdl_wait();
  if (!plan_usable(p, pl)) return;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int G = a.group, cta = blockIdx.x;
  const float scale2 = a.scale * 1.4426950408889634f;
  const int64_t layer_elems = p.layer_bytes() / 4, page_elems = p.page_bytes() / 4,
                head_elems = p.head_bytes() / 4;
  const float* kbase = reinterpret_cast<const float*>(p.k) + a.layer * layer_elems;
  const float* vbase = reinterpret_cast<const float*>(p.v) + a.layer * layer_elems;
  PageItem it;
  for (ItemWalk walk(pl, cta); walk.next(&it);) {
    const int t0 = walk.t0, t1 = walk.t1;
    __syncthreads();  // the previous item's shared tiles are done with
    for (int i = tid; i < M * words; i += kThreads) {
      const int r = i / words, c = i % words, j = r / G;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (j < it.n_rows)
        x = *reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(a.q) + (int64_t)(it.row0 + j) * a.q_stride +
                                            (int64_t)(it.kv_head * G + r % G) * hd + c * E);
      *reinterpret_cast<uint4*>(Qs + r * ld + c * E) = x;
    }
    float m[RM], l[RM], acc[RM][NC];
    int vis[RM];
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      const int j = (ty * RM + i) / G;
      vis[i] = a.causal ? min(max(it.last0 + j + 1, 0), it.n_keys) : it.n_keys;
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[i][c] = 0.f;
    }
    const int32_t* table = p.table + (int64_t)it.seq * p.max_pages;
    for (int t = t0; t < t1; ++t) {
      const int k0 = t * kTile;
      __syncthreads();
      for (int i = tid; i < kTile * words; i += kThreads) {
        const int r = i / words, c = i % words, key = k0 + r;
        uint4 kx = make_uint4(0, 0, 0, 0), vx = kx;
        if (key < it.n_keys) {
          const int page = table[key >> p.page_shift];
          if ((unsigned)page < (unsigned)p.n_pages) {
            const int64_t at = page * page_elems + it.kv_head * head_elems +
                               (int64_t)(key & (p.page_tokens - 1)) * hd + c * E;
            kx = *reinterpret_cast<const uint4*>(kbase + at);
            vx = *reinterpret_cast<const uint4*>(vbase + at);
          } else {
            raise_on_plan(p, pl, ERR_BAD_INDEX, 90);
          }
        }
        *reinterpret_cast<uint4*>(Ks + r * ld + c * E) = kx;
        *reinterpret_cast<uint4*>(Vs + r * hd + c * E) = vx;
      }
      __syncthreads();
      float s[RM][4] = {};
      for (int d = 0; d < hd; d += 4) {
        float4 kv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * j) * ld + d);
#pragma unroll
        for (int i = 0; i < RM; ++i) {
          const float4 qv = *reinterpret_cast<const float4*>(Qs + (ty * RM + i) * ld + d);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s[i][j] = fmaf(qv.x, kv[j].x, fmaf(qv.y, kv[j].y, fmaf(qv.z, kv[j].z, fmaf(qv.w, kv[j].w, s[i][j]))));
        }
      }
#pragma unroll
      for (int i = 0; i < RM; ++i) {
        float mx = m[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = k0 + tx + 16 * j < vis[i] ? s[i][j] * scale2 : -INFINITY;
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float base = mx == -INFINITY ? 0.f : mx;  // no key of this row yet
        const float corr = exp2f(m[i] - base);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float pj = exp2f(s[i][j] - base);
          Ps[(ty * RM + i) * (kTile + 4) + tx + 16 * j] = pj;
          sum += pj;
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[i] = l[i] * corr + sum;
        m[i] = mx;
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[i][c] *= corr;
      }
      __syncwarp();  // a row's scores are written and read by one half-warp
      for (int k = 0; k < kTile; k += 4) {
        float4 pv[RM];
#pragma unroll
        for (int i = 0; i < RM; ++i) pv[i] = *reinterpret_cast<const float4*>(Ps + (ty * RM + i) * (kTile + 4) + k);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          if (c >= nc) break;
          const float* v = Vs + k * hd + tx + 16 * c;
#pragma unroll
          for (int i = 0; i < RM; ++i)
            acc[i][c] = fmaf(pv[i].x, v[0], fmaf(pv[i].y, v[hd], fmaf(pv[i].z, v[2 * hd], fmaf(pv[i].w, v[3 * hd], acc[i][c]))));
        }
      }
      __syncwarp();
    }
    if (!walk.whole(it)) {
      // divided among CTAs: the last to arrive joins the parts
      const int c0 = walk.first_cta(it), c1 = walk.last_cta(it);
      const int part_words = M * (hd + 2);
      float* mine = part_of(pl, part_words, cta, cta == c0);
#pragma unroll
      for (int i = 0; i < RM; ++i) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
          if (c < nc) __stcg(mine + (i * nc + c) * kThreads + tid, acc[i][c]);
        if (tx == 0) {
          __stcg(mine + M * hd + ty * RM + i, m[i]);
          __stcg(mine + M * hd + M + ty * RM + i, l[i]);
        }
      }
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const int n = atomicAdd(&pl.arrived[walk.index], 1);
        s_last = n == c1 - c0;
        if (s_last) pl.arrived[walk.index] = 0;
      }
      __syncthreads();
      if (!s_last) continue;
      __threadfence();
#pragma unroll
      for (int i = 0; i < RM; ++i) {
        const int r = ty * RM + i;
        m[i] = -INFINITY;
        for (int c = c0; c <= c1; ++c) m[i] = fmaxf(m[i], __ldcg(part_of(pl, part_words, c, c == c0) + M * hd + r));
        const float base = m[i] == -INFINITY ? 0.f : m[i];
        l[i] = 0.f;
#pragma unroll
        for (int k = 0; k < NC; ++k) acc[i][k] = 0.f;
        for (int c = c0; c <= c1; ++c) {
          const float* part = part_of(pl, part_words, c, c == c0);
          const float wt = exp2f(__ldcg(part + M * hd + r) - base);
          l[i] = fmaf(wt, __ldcg(part + M * hd + M + r), l[i]);
#pragma unroll
          for (int k = 0; k < NC; ++k)
            if (k < nc) acc[i][k] = fmaf(wt, __ldcg(part + (i * nc + k) * kThreads + tid), acc[i][k]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      const int r = ty * RM + i, j = r / G, h = it.kv_head * G + r % G;
      if (j >= it.n_rows) continue;
      const float inv = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : NAN);  // a row that sees no key gives zeros
      float* dst = reinterpret_cast<float*>(a.o) + (int64_t)(it.row0 + j) * a.o_stride + (int64_t)h * hd;
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (c < nc) dst[tx + 16 * c] = acc[i][c] * inv;
      if (a.lse && tx == 0)
        a.lse[(int64_t)(it.row0 + j) * a.n_q_heads + h] = m[i] == -INFINITY ? -INFINITY : m[i] * 0.6931471805599453f + logf(l[i]);
    }
  }
}

namespace {

template <int M, int NC>
cudaError_t launch_simt(const PagesView& p, const PagesPlan& pl, const AttnArgs& a, cudaStream_t s) {
  const size_t smem = 4 * (size_t)(M * (p.head_dim + 4) + kTile * (p.head_dim + 4) + kTile * p.head_dim + M * (kTile + 4));
  cudaError_t e = cudaFuncSetAttribute(attention_simt_kernel<M, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024);
  if (e != cudaSuccess) return e;
  return launch_ex(attention_simt_kernel<M, NC>, dim3(pl.ctas), dim3(kThreads), smem, s, true, p, pl, a);
}

template <int M>
cudaError_t simt_dim(const PagesView& p, const PagesPlan& pl, const AttnArgs& a, cudaStream_t s) {
  if (p.head_dim <= 64) return launch_simt<M, 4>(p, pl, a, s);
  if (p.head_dim <= 128) return launch_simt<M, 8>(p, pl, a, s);
  return launch_simt<M, 16>(p, pl, a, s);
}

}  // namespace

cudaError_t pages_attention_simt(const PagesView& p, const PagesPlan& pl, const AttnArgs& a, bool few, cudaStream_t s) {
  return few ? simt_dim<16>(p, pl, a, s) : simt_dim<64>(p, pl, a, s);
}

}  // namespace duolm
