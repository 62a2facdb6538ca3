// The router: each token's k experts, their weights, and the order that
// sorts the (token, choice) pairs by expert.
//
//   valid_i = l_i > -inf (NaN counts as -inf, +inf as the largest float)
//   ids     = the k largest valid logits, largest first, ties to the lowest i
//   w_j     = exp(l_j - m) / sum over the valid (or, renormalised, over the
//             chosen) of exp(l - m), m the largest logit
//   row of (t, j) = rows of lower experts + earlier tokens with this expert
//
// A group of L lanes takes a token, V = 8 or 16 consecutive logits a lane
// (L = 4 to 32 by E).  Each lane sorts its own once, by eights (sixteen at once
// went to local memory: 70 us for 11000 tokens of 280); a choice is then the
// largest of the lanes' heads, found in log2(L) exchanges, and the lane that
// has it (the lowest of equals: lanes hold rising indices) drops its head.
// Tokens are dealt to CTAs in chunks.  In a chunk each expert has a bit per
// token, set by whoever chose it: a population count below a token's bit is
// its place among the chunk's rows of that expert, in token order and without
// any order of the setting.  The chunks' counts go to a small matrix; a
// second kernel adds to each place the rows of the chunks before and of the
// lower experts; when there are more chunks than SMs a kernel between the two
// sums the matrix once.  A single chunk does all in one launch.
// The logits are read once (4 bytes x E a token), but the choices' compares
// and selects bound it: 65536 tokens, 8 of 128 experts, 29 us for the choices
// where the logits' 34 MB take 5, 12 for the rows, 13 for the gradient.  For
// few tokens it is one launch (64 tokens, 8 of 64: 4.7 us); a million tokens,
// 8 of 128, take 504 us.
#include <mutex>
#include <type_traits>

#include "route.cuh"

namespace bra {
namespace {

using namespace route;

// The experts of one token to each group of L lanes (t < 0: none); lane l of
// the group holds logits l * V ..  Writes ids and weights and sets the
// chunk's bits (word `word`, bit `bit` of each expert's `stride`).  Whole warps.
template <typename T, int L, int V>
__device__ __forceinline__ void choose(const RouteParams& p, int t, int lane, uint32_t* bits,
                                       int stride, int word, uint32_t bit) {
  constexpr int OWN = (BRA_MAX_CHOICES + L - 1) / L;   // choices a lane keeps
  const int gl = lane % L;
  const uint32_t group = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << (lane & ~(L - 1));
  const T* row = static_cast<const T*>(p.logits) + (int64_t)t * p.E;
  // lists of eight, so that sorting stays short: the lower indices first
  constexpr int NL = V / 8;
  uint32_t key[NL][8], order[NL];               // order: sorted places, four bits each
#pragma unroll
  for (int l = 0; l < NL; ++l) {
    int idx[8];
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const int at = gl * V + l * 8 + i;
      T raw[4];
      if (t >= 0 && p.vec && at + 4 <= p.E) {
        if constexpr (sizeof(T) == 4)
          *reinterpret_cast<uint4*>(raw) = *reinterpret_cast<const uint4*>(row + at);
        else
          *reinterpret_cast<uint2*>(raw) = *reinterpret_cast<const uint2*>(row + at);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) raw[c] = t >= 0 && at + c < p.E ? row[at + c] : T(-INFINITY);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        key[l][i + c] = key_of(logit(&raw[c]));
        idx[i + c] = i + c;
      }
    }
    sort_eight(key[l], idx);
    order[l] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) order[l] |= (uint32_t)idx[i] << (4 * i);
  }
  uint32_t my_key[OWN], top = 0u;
  int my_id[OWN];
#pragma unroll
  for (int o = 0; o < OWN; ++o) {
    my_key[o] = 0u;
    my_id[o] = -1;
    for (int j = o * L; j < min(p.k, (o + 1) * L); ++j) {
      uint32_t head = key[0][0];
      int from = 0, place = (int)(order[0] & 15u);
      if (NL == 2 && key[NL - 1][0] > head) {
        head = key[NL - 1][0];
        from = 1;
        place = 8 + (int)(order[NL - 1] & 15u);
      }
      uint32_t most = head;
#pragma unroll
      for (int d = L / 2; d > 0; d >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
      const uint32_t has = __ballot_sync(0xffffffffu, head == most) & group;
      const int win = __ffs(has) - 1;
      const int at = __shfl_sync(0xffffffffu, gl * V + place, win);
      if (j == 0) top = most;
      if (gl == j - o * L && most) {
        my_key[o] = most;
        my_id[o] = at;
      }
      // the winner drops its head (with most = 0 there is nothing to drop)
#pragma unroll
      for (int l = 0; l < NL; ++l) {
        const bool drop = lane == win && from == l;
#pragma unroll
        for (int i = 0; i + 1 < 8; ++i) key[l][i] = drop ? key[l][i + 1] : key[l][i];
        key[l][7] = drop ? 0u : key[l][7];
        order[l] = drop ? order[l] >> 4 : order[l];
      }
    }
  }
  const float m = value_of(top);
  float e[OWN], s = 0.f;
#pragma unroll
  for (int o = 0; o < OWN; ++o) {
    e[o] = my_key[o] ? expf(value_of(my_key[o]) - m) : 0.f;
    s += e[o];
  }
  if (!p.renorm) {
    // all open logits: the ones left, and the chosen
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i / 8][i % 8]) s += expf(value_of(key[i / 8][i % 8]) - m);
  }
  s = group_sum(s, L);
  const int64_t out = (int64_t)t * p.k;
#pragma unroll
  for (int o = 0; o < OWN; ++o)
    if (t >= 0 && o * L + gl < p.k) {
      p.ids[out + o * L + gl] = my_id[o];
      p.weights[out + o * L + gl] = my_key[o] ? e[o] / s : 0.f;
      if (my_id[o] >= 0) atomicOr(&bits[my_id[o] * stride + word], bit);
    }
}

template <typename T, int L, int V>
__global__ void __launch_bounds__(kThreads) route_choose_kernel(const RouteParams p) {
  extern __shared__ uint32_t bits[];                    // [E][stride]
  clear_bits(bits, p.E * bit_stride(p.chunk));
  __syncthreads();
  grid_wait();
  grid_go();
  route_chunk_of<L>(p, bits, [&](int t, int lane, int stride, int word, uint32_t bit) {
    choose<T, L, V>(p, t, lane, bits, stride, word, bit);
  });
}

// The matrix of counts, summed down its columns in place: a CTA to 32 experts,
// 32 chunks at a time, each expert's by one warp.
__global__ void __launch_bounds__(kThreads) route_scan_kernel(const RouteParams p) {
  __shared__ int tile[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + lane;
  auto load = [&](int r) {
    return e < p.E && r < p.chunks ? p.hist[(int64_t)r * p.E + e] : 0;
  };
  grid_wait();
  grid_go();
  int carry = 0, next = load(warp);
  for (int r0 = 0; r0 < p.chunks; r0 += 32) {
    tile[warp][lane] = next;                 // a warp holds a chunk, a lane an expert
    next = load(r0 + 32 + warp);
    __syncthreads();
    int v = tile[lane][warp];                // the other way round
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += a;
    }
    v += carry;
    carry = __shfl_sync(0xffffffffu, v, 31);
    tile[lane][warp] = v;                    // read by this thread alone until here
    __syncthreads();
    if (e < p.E && r0 + warp < p.chunks) p.hist[(int64_t)(r0 + warp) * p.E + e] = tile[warp][lane];
    // the next round's write goes to the element this thread has just read
  }
}

// Rows of one chunk, from the counts of all of them, or from their sums.
__global__ void __launch_bounds__(kThreads) route_place_kernel(const RouteParams p) {
  __shared__ int total[kMaxGroups], before[kMaxGroups], base[kMaxGroups];
  __shared__ int used;
  const int c = blockIdx.x, t0 = c * p.chunk;
  const int n = min(p.chunk, p.T - t0);
  for (int e = threadIdx.x; e < p.E; e += kThreads) total[e] = before[e] = 0;
  __syncthreads();
  grid_wait();                                          // the choices are written
  grid_go();
  // the first pairs' loads go out before the matrix is summed
  constexpr int AHEAD = 4;
  int id[AHEAD], place[AHEAD];
#pragma unroll
  for (int a = 0; a < AHEAD; ++a) {
    const int i = threadIdx.x + a * kThreads;
    const bool in = i < n * p.k;
    id[a] = in ? p.ids[(int64_t)t0 * p.k + i] : -1;
    place[a] = in ? p.slots[(int64_t)t0 * p.k + i] : -1;
  }
  // threads of a row of the matrix side by side, rows dealt over the rest
  const int width = (p.E + 31) / 32 * 32, rows = kThreads / width;
  const int e = threadIdx.x % width, r0 = threadIdx.x / width;
  if (p.scanned) {
    for (int i = threadIdx.x; i < p.E; i += kThreads) {
      total[i] = p.hist[(int64_t)(p.chunks - 1) * p.E + i];
      before[i] = c ? p.hist[(int64_t)(c - 1) * p.E + i] : 0;
    }
  } else if (e < p.E && r0 < rows) {
    int all = 0, old = 0;
#pragma unroll 16
    for (int r = r0; r < p.chunks; r += rows) {
      const int h = p.hist[(int64_t)r * p.E + e];
      all += h;
      old += r < c ? h : 0;
    }
    atomicAdd(&total[e], all);
    atomicAdd(&before[e], old);
  }
  __syncthreads();
  scan_experts(p, total, before, base, &used);
  if (c == 0)
    for (int i = threadIdx.x; i < p.E; i += kThreads) p.counts[i] = total[i];
  auto put = [&](int i, int e1, int at) {
    if (e1 >= 0) {
      const int slot = at + base[e1];
      p.slots[(int64_t)t0 * p.k + i] = slot;
      p.tokens[slot] = t0 + i / p.k;
    }
  };
#pragma unroll
  for (int a = 0; a < AHEAD; ++a) put(threadIdx.x + a * kThreads, id[a], place[a]);
  for (int i = threadIdx.x + AHEAD * kThreads; i < n * p.k; i += kThreads)
    put(i, p.ids[(int64_t)t0 * p.k + i], p.slots[(int64_t)t0 * p.k + i]);
  mark_unused(p, c, used);
}

// --------------------------------------------------------------------------
// Gradient of the logits: with g the gradient of the weights and s = sum w g,
//   renormalised:  dl_i = w_j (g_j - s) for the chosen i = id_j, else 0
//   otherwise:     dl_i = p_i ([i = id_j] g_j - s), p the softmax
// Weights that were multiplied by c: w and s are c times as large, and g_j
// loses s / c.  Sigmoid scores: the chosen ones' dl_i times 1 - sigmoid(l_i),
// with s = 0 when not renormalised.
// --------------------------------------------------------------------------
struct RouteGradParams {
  const float* dweights;
  const void* logits;
  const int32_t* ids;
  const float* weights;
  void* dlogits;
  int T, E, k, renorm;
  int vec;             // rows are written four at a time
  int sigmoid;
  float inv_scale;     // one over what the weights were multiplied by
};

template <typename T>
__device__ __forceinline__ T rounded(float v) {
  return static_cast<T>(v);
}

// A group of L lanes takes a token: the row is written whole as if nothing
// were chosen, four elements a store, then the chosen ones over it (p_i is
// w_j there).
template <typename T, int L, int V>
__global__ void __launch_bounds__(256) route_grad_kernel(const RouteGradParams p) {
  constexpr int G = 32 / L, OWN = (BRA_MAX_CHOICES + L - 1) / L;
  const int lane = threadIdx.x & 31, gl = lane % L;
  grid_wait();
  grid_go();
  const int64_t step = (int64_t)gridDim.x * 8 * G;
  const int64_t first = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * G;
  int id[OWN], id_next[OWN];
  float w[OWN], g[OWN], w_next[OWN], g_next[OWN];
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
      const int j = o * L + gl;
      const bool have = t < p.T && j < p.k;
      id_next[o] = have ? p.ids[t * p.k + j] : -1;
      w_next[o] = have ? p.weights[t * p.k + j] : 0.f;
      g_next[o] = have ? p.dweights[t * p.k + j] : 0.f;
    }
  };
  fetch(first + lane / L);
  for (int64_t t0 = first; t0 < p.T; t0 += step) {
    const int64_t t = t0 + lane / L;
    const bool in = t < p.T;
    float s = 0.f;
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
      const bool open = id_next[o] >= 0 && id_next[o] < p.E;
      id[o] = open ? id_next[o] : -1;
      w[o] = open ? w_next[o] : 0.f;
      g[o] = open ? g_next[o] : 0.f;
      s += w[o] * g[o];
    }
    fetch(t + step);
    s = group_sum(s, L);
    float d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = 0.f;
    float rest[OWN];                 // 1 - sigmoid of the chosen logits
#pragma unroll
    for (int o = 0; o < OWN; ++o) rest[o] = 1.f;
    const T* row = static_cast<const T*>(p.logits) + t * p.E;
    if (p.sigmoid) {
#pragma unroll
      for (int o = 0; o < OWN; ++o)
        if (id[o] >= 0) rest[o] = 1.f / (1.f + expf(logit(row + id[o])));
    } else if (!p.renorm) {
      uint32_t best = 0u;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        d[i] = in && gl * V + i < p.E ? logit(row + gl * V + i) : -INFINITY;
        best = max(best, key_of(d[i]));
      }
#pragma unroll
      for (int m = L / 2; m > 0; m >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, m));
      const float m = value_of(best);
      float sum = 0.f;
      uint32_t open = 0u;            // bit i: whether this lane's logit i is open
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const bool is = key_of(d[i]) != 0u;
        open |= (is ? 1u : 0u) << i;
        d[i] = is ? expf(d[i] - m) : 0.f;
        sum += d[i];
      }
      sum = group_sum(sum, L);
      const float f = sum > 0.f ? -s / sum : 0.f;
      // a closed expert gets 0 whatever f is: 0 times an infinite s is NaN
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = (open >> i) & 1u ? d[i] * f : 0.f;
    }
    T* out = static_cast<T*>(p.dlogits) + t * p.E;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const int at = gl * V + i;
      T r[4] = {rounded<T>(d[i]), rounded<T>(d[i + 1]), rounded<T>(d[i + 2]), rounded<T>(d[i + 3])};
      if (in && p.vec && at + 4 <= p.E) {
        if constexpr (sizeof(T) == 4)
          *reinterpret_cast<uint4*>(out + at) = *reinterpret_cast<const uint4*>(r);
        else
          *reinterpret_cast<uint2*>(out + at) = *reinterpret_cast<const uint2*>(r);
      } else if (in) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (at + c < p.E) out[at + c] = r[c];
      }
    }
    __syncwarp();                    // the row lies before its chosen elements are written
    const float mean = p.sigmoid && !p.renorm ? 0.f : s * p.inv_scale;
#pragma unroll
    for (int o = 0; o < OWN; ++o)
      if (id[o] >= 0) out[id[o]] = rounded<T>(w[o] * (g[o] - mean) * rest[o]);
    __syncwarp();
  }
}

// f for the logits' type, the lanes of a token and the logits of a lane.
template <typename F>
cudaError_t by_type(int dtype, int E, F&& f) {
  auto by_lanes = [&](auto* type) {
    using std::integral_constant;
    if (E <= 32) return f(type, integral_constant<int, 4>{}, integral_constant<int, 8>{});
    if (E <= 64) return f(type, integral_constant<int, 8>{}, integral_constant<int, 8>{});
    if (E <= 128) return f(type, integral_constant<int, 16>{}, integral_constant<int, 8>{});
    if (E <= 256) return f(type, integral_constant<int, 32>{}, integral_constant<int, 8>{});
    return f(type, integral_constant<int, 32>{}, integral_constant<int, 16>{});
  };
  if (dtype == BRA_FP32) return by_lanes((float*)nullptr);
  if (dtype == BRA_BF16) return by_lanes((__nv_bfloat16*)nullptr);
  return by_lanes((__half*)nullptr);
}

// Lets the kernel have the shared memory of its largest call, once a device.
// The limit belongs to the kernel, not to a call: set to a call's own size it
// could be lowered between another thread's setting and its launch.
template <typename T, int L, int V>
cudaError_t choose_ready() {
  constexpr int most = (L * V < kMaxGroups ? L * V : kMaxGroups) * bit_stride(kMostChunk) * 4;
  static std::mutex mu;
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  if (!ready[dev & 63]) {
    e = cudaFuncSetAttribute(route_choose_kernel<T, L, V>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    ready[dev & 63] = true;
  }
  return cudaSuccess;
}

}  // namespace

// Tokens of a chunk: one chunk up to 64 tokens (one launch); else chunks of at
// most kMostChunk tokens, as many for each of 152 SMs.
int route_chunk(int64_t T) {
  if (T <= 64) return 64;
  const int64_t chunks = (T + 152 * kMostChunk - 1) / (152 * kMostChunk) * 152;
  return (int)(((T + chunks - 1) / chunks + 31) / 32 * 32);
}

// Chunks from which the counts are summed by a launch of their own.  Below,
// each CTA of the last kernel sums the matrix itself, in all the square of the
// chunks.  8 of 128 experts, us, by each CTA / by the launch: 65536 tokens (147
// chunks) 35.1 / 35.8, 262144 (304) 132 / 129, 1048576 (1058) 576 / 504,
// 4194304 (4096) 3045 / 1982.
constexpr int kScanChunks = 160;

void route_chunks(RouteParams* p) {
  p->chunk = route_chunk(p->T);
  p->chunks = (int)(((int64_t)p->T + p->chunk - 1) / p->chunk);
  p->scanned = p->chunks >= kScanChunks;
}

cudaError_t launch_route_places(const RouteParams& p, cudaStream_t st) {
  if (p.chunks == 1) return cudaSuccess;
  if (p.scanned) {
    const cudaError_t a =
        launch_overlapped(route_scan_kernel, (unsigned)(p.E + 31) / 32, kThreads, 0, st, p);
    if (a != cudaSuccess) return a;
  }
  return launch_overlapped(route_place_kernel, (unsigned)p.chunks, kThreads, 0, st, p);
}

cudaError_t launch_route(const RouteCall& r, cudaStream_t st) {
  RouteParams p = {r.logits, r.ids, r.weights, r.counts, r.slots, r.tokens, r.hist, (int)r.T,
                   r.E,      r.k,   r.renorm,  0,        0,       rows_vec(r.logits, r.E, r.dtype), 0};
  route_chunks(&p);
  const int smem = r.E * bit_stride(p.chunk) * 4;
  const cudaError_t e = by_type(r.dtype, r.E, [&](auto* type, auto l, auto v) {
    using T = std::remove_pointer_t<decltype(type)>;
    const cudaError_t a = choose_ready<T, decltype(l)::value, decltype(v)::value>();
    if (a != cudaSuccess) return a;
    return launch_overlapped(route_choose_kernel<T, decltype(l)::value, decltype(v)::value>,
                             (unsigned)p.chunks, kThreads, smem, st, p);
  });
  return e != cudaSuccess ? e : launch_route_places(p, st);
}

cudaError_t launch_route_grad(const RouteGradCall& r, cudaStream_t st) {
  const RouteGradParams p = {r.dweights, r.logits, r.ids, r.weights, r.dlogits,
                             (int)r.T,   r.E,      r.k,   r.renorm,
                             rows_vec(r.dlogits, r.E, r.dtype), r.sigmoid, 1.f / r.scale};
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  return by_type(r.dtype, r.E, [&](auto* type, auto l, auto v) {
    using T = std::remove_pointer_t<decltype(type)>;
    constexpr int tokens = 8 * 32 / decltype(l)::value;           // of a block
    const int64_t want = (r.T + tokens - 1) / tokens, full = (int64_t)sms * 8;
    return launch_overlapped(route_grad_kernel<T, decltype(l)::value, decltype(v)::value>,
                             (unsigned)(want < full ? want : full), 256, 0, st, p);
  });
}

}  // namespace bra
