// Tokens sorted by expert and back, for experts of the caller's own, with the gradients of
// both moves and of the top-k weights.
//
// With N = T k assignments a = t k + j of keys e_a (the expert, or E for an index outside
// [0, E), an assignment that is dropped):
//   place(a) = #{b : (e_b, b) < (e_a, a)}          a stable counting sort
//   rows[place(a)] = x[t]                          0 where dropped
//   out[t] = sum_j w[t, j] y[place(t, j)]          and its gradients
//   dy[place(t, j)] = w[t, j] dout[t],  dw[t, j] = <dout[t], y[place(t, j)]>
// Everything but the dot products and the sums over j is movement: bound by memory.
#include "moe_dense.cuh"
#include "sm100_ptx.cuh"

namespace moe {

namespace {

constexpr int kKeys = kMaxExperts + 1;  // the experts, and what is dropped
constexpr uint64_t kLandingNs = 20000000ull;  // after a wait that gave up: in this time every issued copy has landed (20 ms)

__device__ uint32_t g_sort_status;  // bits as in the layer's status word

__device__ __forceinline__ int key_of(int e, int E) { return e >= 0 && e < E ? e : E; }

// ------------------------------------------------------------------ many assignments: the order
// By one cluster.  Each warp takes a contiguous run of assignments and counts their keys, which
// gives each its rank among its key's in the run; the blocks tell one another their sums, from
// which each knows where its keys begin.  What bounds it is the latency of these few steps,
// which the rows' copies of the next launch hide in part: it starts with this one and has its
// first rows in before the order is there.  Up to kHeld x 32 assignments of a run stay in
// registers; a second reading of them, a load and a match at a time, took 2 of 8 us at 16384
// assignments and 8 of 15 at 65536.
constexpr int kOrderThreads = 1024, kOrderWarps = kOrderThreads / 32, kOrderBlocks = 8, kHeld = 8;

__global__ void __cluster_dims__(kOrderBlocks, 1, 1) __launch_bounds__(kOrderThreads)
    order_kernel(const __grid_constant__ SortParams p) {
  __shared__ int count[kOrderWarps][kKeys + 2];
  __shared__ int sums[kOrderBlocks][kKeys + 3];  // written by every block of the cluster
  __shared__ int first[kKeys];
  __shared__ int warp_total[kOrderWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, keys = p.E + 1, rank = blockIdx.x;
  for (int i = tid; i < kOrderWarps * (kKeys + 2); i += kOrderThreads) (&count[0][0])[i] = 0;
  __syncthreads();
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  ptx::cluster_arrive_release();  // (every block has started: its memory may be written)
  const int n = p.T * p.k, warps = kOrderBlocks * kOrderWarps, run = ceil_div(ceil_div(n, warps), 32) * 32;
  const int begin = min(n, (rank * kOrderWarps + warp) * run), end = min(n, begin + run);
  const int bits = 32 - __clz(p.E);  // of a key
  int* const own = count[warp];
  // the keys of 32 kHeld assignments from `a0` on, -1 past the run's end
  int key[kHeld], at[kHeld];
  auto load = [&](int a0) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int a = a0 + 32 * i + lane;
      key[i] = a < end ? key_of(__ldcg(p.idx + a), p.E) : -1;
    }
  };
  // their ranks in the run, and the run's counts so far
  auto ranks = [&](int a0) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      if (a0 + 32 * i >= end) break;
      // the lanes of the same key, by a vote for each of its bits (one match instruction for it took
      // the SM about 50 cycles: 65536 assignments 14.3 us)
      unsigned same = __ballot_sync(0xffffffffu, key[i] >= 0);
      for (int b = 0; b < bits; ++b) {
        const bool set = key[i] >> b & 1;
        const unsigned vote = __ballot_sync(0xffffffffu, set);
        same &= set ? vote : ~vote;
      }
      const int ahead = __popc(same & ((1u << lane) - 1));
      const int before = key[i] >= 0 ? own[key[i]] : 0;
      at[i] = before + ahead;
      __syncwarp();
      if (key[i] >= 0 && ahead == 0) own[key[i]] = before + __popc(same);
      __syncwarp();
    }
  };
  const bool held = run <= 32 * kHeld;
  if (held) {
    load(begin);
    ranks(begin);
  } else {
    for (int a0 = begin; a0 < end; a0 += 32 * kHeld) {
      load(a0);
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (key[i] >= 0) atomicAdd(&own[key[i]], 1);
    }
  }
  __syncthreads();
  // a warp's places of a key begin behind those of the lower warps
  int total = 0;
  if (tid < keys) {
    int c[kOrderWarps];
#pragma unroll
    for (int w = 0; w < kOrderWarps; ++w) c[w] = count[w][tid];
#pragma unroll
    for (int w = 0; w < kOrderWarps; ++w) {
      count[w][tid] = total;
      total += c[w];
    }
  }
  __syncwarp();
  ptx::cluster_wait_acquire();
  if (tid < keys) {
    const uint32_t mine = ptx::smem_u32(&sums[rank][tid]);
#pragma unroll
    for (int b = 0; b < kOrderBlocks; ++b)
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(ptx::mapa_shared(mine, b)), "r"(total) : "memory");
  }
  __syncwarp();
  ptx::cluster_arrive_release();
  ptx::cluster_wait_acquire();
  // behind the lower blocks', and all of them behind those of the lower keys
  int before = 0, all = 0;
  if (tid < keys) {
#pragma unroll
    for (int b = 0; b < kOrderBlocks; ++b) {
      const int s = sums[b][tid];
      if (b < rank) before += s;
      all += s;
    }
  }
  int scan = all;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, scan, d);
    if (lane >= d) scan += o;
  }
  if (lane == 31) warp_total[warp] = scan;
  __syncthreads();
  if (tid < keys) {
    int to = scan - all;
    for (int w = 0; w < warp; ++w) to += warp_total[w];
    first[tid] = to + before;
    if (rank == 0) p.offsets[tid] = to;
  }
  __syncthreads();
  auto place = [&](int a0) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int a = a0 + 32 * i + lane;
      if (key[i] < 0) continue;
      const int to = first[key[i]] + at[i] + (held ? own[key[i]] : 0);
      p.inv_perm[a] = key[i] < p.E ? to : -1 - to;
    }
  };
  if (held) {
    place(begin);
  } else {  // (the run's first places, counted on from)
    for (int a0 = begin; a0 < end; a0 += 32 * kHeld) {
      load(a0);
      ranks(a0);
      place(a0);
    }
  }
}

// A token's scales to the places of its assignments (zeros to those of dropped ones), by a
// warp: read once, four units a lane at a time.  place(j): as in inv_perm, the same in every lane.
template <typename U, typename Place>
__device__ __forceinline__ void move_units(const SortParams& p, size_t t, Place place) {
  constexpr int kAtOnce = 4;
  const int units = p.scale_bytes / (int)sizeof(U), lane = threadIdx.x & 31;
  const U* from = reinterpret_cast<const U*>(p.scales) + t * units;
  for (int i0 = 0; i0 < units; i0 += 32 * kAtOnce) {
    U held[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (i0 + 32 * i + lane < units) held[i] = __ldcg(from + i0 + 32 * i + lane);
    for (int j = 0; j < p.k; ++j) {
      const int at = place(j);
      U* to = reinterpret_cast<U*>(p.row_scales) + (size_t)(at >= 0 ? at : -1 - at) * units;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (i0 + 32 * i + lane < units) to[i0 + 32 * i + lane] = at >= 0 ? held[i] : U(0);
    }
  }
}
template <typename Place>
__device__ __forceinline__ void move_scales(const SortParams& p, size_t t, Place place) {
  // (the widest unit that the rows' length and both arrays' beginnings are multiples of)
  const unsigned bits = (unsigned)p.scale_bytes | (unsigned)reinterpret_cast<uintptr_t>(p.scales) |
                        (unsigned)reinterpret_cast<uintptr_t>(p.row_scales);
  if ((bits & 3) == 0)
    move_units<unsigned>(p, t, place);
  else if ((bits & 1) == 0)
    move_units<unsigned short>(p, t, place);
  else
    move_units<unsigned char>(p, t, place);
}

// Zeros to a dropped assignment's row, by a warp.
__device__ __forceinline__ void zero_row(const SortParams& p, size_t at) {
  uint4* row = reinterpret_cast<uint4*>(p.rows) + at * (p.row_bytes / 16);
  for (int v = threadIdx.x & 31; v < p.row_bytes / 16; v += 32) row[v] = make_uint4(0, 0, 0, 0);
}

// The rows: each warp takes tokens in turn, whose rows come to its ring in shared memory by one
// bulk copy and leave it by one for each of their places, issued by as many lanes.  The rows
// are asked for before the order of the launch before is there.  (x was complete when that
// launch passed its own wait, before which this one cannot start.)
constexpr int kGatherStages = 2;
__global__ void __launch_bounds__(128) gather_kernel(const __grid_constant__ SortParams p) {
  extern __shared__ __align__(128) uint8_t gather_smem[];
  __shared__ uint64_t full_bar[4][kGatherStages];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  uint8_t* const ring = gather_smem + (size_t)warp * kGatherStages * p.row_bytes;
  uint64_t* const bar = full_bar[warp];
  const uint8_t* x = reinterpret_cast<const uint8_t*>(p.x);
  uint8_t* rows = reinterpret_cast<uint8_t*>(p.rows);
  const int t0 = blockIdx.x * warps + warp, step = gridDim.x * warps;
  auto issue = [&](int s, int t) {
    ptx::mbar_arrive_expect_tx(&bar[s], p.row_bytes);
    ptx::bulk_load(ring + (size_t)s * p.row_bytes, x + (size_t)t * p.row_bytes, p.row_bytes, &bar[s]);
  };
  if (lane == 0) {
    for (int s = 0; s < kGatherStages; ++s) ptx::mbar_init(&bar[s], 1);
    ptx::fence_mbar_init();
    for (int s = 0; s < kGatherStages; ++s)
      if ((long long)t0 + (long long)s * step < p.T) issue(s, t0 + s * step);
  }
  __syncwarp();
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  int s = 0;
  uint32_t phase = 0;
  bool ok = true;
  int next = t0 < p.T && lane < p.k ? __ldcg(p.inv_perm + (size_t)t0 * p.k + lane) : 0;
  for (long long t = t0; t < p.T; t += step) {
    const int at = next;
    if (t + step < p.T && lane < p.k) next = __ldcg(p.inv_perm + (size_t)(t + step) * p.k + lane);
    if (ok && !ptx::mbar_wait_bounded(&bar[s], phase, p.wait_ns)) ok = false;
    ok = __all_sync(0xffffffffu, ok);
    const bool on = lane < p.k;
    if (on) {  // (here, where every SM writes, and not by the few that found the order)
      const int a = (int)t * p.k + lane;
      p.perm[at >= 0 ? at : -1 - at] = at >= 0 ? a : -1 - a;
    }
    if (on && at >= 0 && ok) {
      ptx::bulk_store(rows + (size_t)at * p.row_bytes, ring + (size_t)s * p.row_bytes, p.row_bytes);
      ptx::bulk_commit();
    }
    unsigned gone = __ballot_sync(0xffffffffu, on && at < 0);
    for (; gone; gone &= gone - 1) zero_row(p, -1 - __shfl_sync(0xffffffffu, at, __ffs(gone) - 1));
    if (p.scale_bytes) move_scales(p, t, [&](int j) { return __shfl_sync(0xffffffffu, at, j); });
    if (on) ptx::bulk_wait_read();
    __syncwarp();
    if (lane == 0 && ok && t + (long long)kGatherStages * step < p.T) issue(s, (int)(t + kGatherStages * step));
    if (++s == kGatherStages) {
      s = 0;
      phase ^= 1;
    }
  }
  ptx::bulk_wait_all();
  // a copy waited for in vain may still land: report, and stay until it surely has
  if (!ok && lane == 0) {
    report_status(&g_sort_status, kStatusTimeoutMain);
    const uint64_t since = ptx::globaltimer_ns();
    while (ptx::globaltimer_ns() - since < kLandingNs) __nanosleep(1000);
  }
}

// ------------------------------------------------------------------ few assignments
// One launch: a block per token finds its assignments' places by counting those before them,
// all N of them for each, while its row comes in.  The last block finds the offsets.  The counting
// grows with T N: 512 x 4 tokens x 2880 4.7 us (by two launches 6.2), 1024 x 4 11.2 (8.1); 2000 x
// 1 x 4096 9.4 (8.5).  Few tokens are bound by the launch and two memory round trips (64 x 4: 2.2).
constexpr int kFewAssignments = 2048, kFewThreads = 128, kFewHeld = 4;
__global__ void __launch_bounds__(kFewThreads) sort_few_kernel(const __grid_constant__ SortParams p) {
  __shared__ __align__(16) uint32_t order[kFewAssignments];  // (key, place) as one number
  __shared__ int place[kMaxTopK];
  __shared__ int count[kKeys + 31];
  const int n = p.T * p.k, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool last = (int)blockIdx.x == p.T;
  const size_t t = blockIdx.x;
  const int vecs = p.row_bytes / 16;
  const uint4* x = reinterpret_cast<const uint4*>(p.x) + t * vecs;
  uint4 held[kFewHeld];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  if (!last) {
#pragma unroll
    for (int i = 0; i < kFewHeld; ++i)
      if (tid + i * kFewThreads < vecs) held[i] = __ldcg(x + tid + i * kFewThreads);
  } else {
    for (int i = tid; i < kKeys + 31; i += kFewThreads) count[i] = 0;
  }
  const int padded = (n + 127) / 128 * 128;
  for (int a = tid; a < padded; a += kFewThreads)
    order[a] = a < n ? (uint32_t)key_of(__ldcg(p.idx + a), p.E) << 16 | (uint32_t)a : 0xFFFFFFFFu;
  __syncthreads();
  if (last) {
    for (int a = tid; a < n; a += kFewThreads) atomicAdd(&count[order[a] >> 16], 1);
    __syncthreads();
    if (warp == 0) {
      int before = 0;
      for (int e0 = 0; e0 <= p.E; e0 += 32) {
        int scan = count[e0 + lane];
        const int own = scan;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, scan, d);
          if (lane >= d) scan += o;
        }
        if (e0 + lane <= p.E) p.offsets[e0 + lane] = before + scan - own;
        before += __shfl_sync(0xffffffffu, scan, 31);
      }
    }
    return;
  }
  for (int j = warp; j < p.k; j += kFewThreads / 32) {
    const int a = (int)t * p.k + j;
    const uint32_t mine = order[a];
    int less = 0;
    for (int b = 4 * lane; b < padded; b += 128) {
      const uint4 o = *reinterpret_cast<const uint4*>(order + b);
      less += (o.x < mine) + (o.y < mine) + (o.z < mine) + (o.w < mine);
    }
    less = __reduce_add_sync(0xffffffffu, less);
    const bool kept = (int)(mine >> 16) < p.E;
    if (lane == 0) {
      place[j] = kept ? less : -1 - less;
      p.perm[less] = kept ? a : -1 - a;
      p.inv_perm[a] = kept ? less : -1 - less;
    }
  }
  __syncthreads();
  uint4* rows = reinterpret_cast<uint4*>(p.rows);
  auto put = [&](int v, const uint4& r) {
    for (int j = 0; j < p.k; ++j) {
      const int at = place[j];
      rows[(size_t)(at >= 0 ? at : -1 - at) * vecs + v] = at >= 0 ? r : make_uint4(0, 0, 0, 0);
    }
  };
#pragma unroll
  for (int i = 0; i < kFewHeld; ++i)
    if (tid + i * kFewThreads < vecs) put(tid + i * kFewThreads, held[i]);
  for (int v = tid + kFewHeld * kFewThreads; v < vecs; v += kFewThreads) put(v, __ldcg(x + v));
  if (p.scale_bytes && warp == 0) move_scales(p, t, [&](int j) { return place[j]; });
}

// ------------------------------------------------------------------ back to tokens
// The row at an entry of inv_perm, or -1 for a dropped assignment's and for one beyond the rows.
__device__ __forceinline__ int row_of(int at, int n) { return at >= 0 && at < n ? at : -1; }

// Few tokens: a block for each, a thread for eight columns of it at a time, loads of this many
// rows in flight together.
constexpr int kRowsAhead = 4;

// out[t] = sum_j w[t, j] y[place(t, j)]
template <typename A>
__global__ void __launch_bounds__(512) unsort_kernel(const __grid_constant__ UnsortParams p) {
  __shared__ int row[kMaxTopK];
  __shared__ float weight[kMaxTopK];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const size_t t = blockIdx.x;
  const int vecs = p.H / 8, tid = threadIdx.x;
  if (tid < p.k) {
    row[tid] = row_of(__ldcg(p.inv_perm + t * p.k + tid), p.T * p.k);
    weight[tid] = p.w ? __ldcg(p.w + t * p.k + tid) : 1.f;
  }
  __syncthreads();
  for (int v = tid; v < vecs; v += blockDim.x) {
    float sum[8] = {};
    for (int j0 = 0; j0 < p.k; j0 += kRowsAhead) {
      Vec8<A> r[kRowsAhead];
#pragma unroll
      for (int j = 0; j < kRowsAhead; ++j)
        if (j0 + j < p.k && row[j0 + j] >= 0) r[j].load(p.y, (size_t)row[j0 + j] * vecs + v);
#pragma unroll
      for (int j = 0; j < kRowsAhead; ++j) {
        if (j0 + j >= p.k || row[j0 + j] < 0) continue;
        float f[8];
        r[j].get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = fmaf(weight[j0 + j], f[i], sum[i]);
      }
    }
    Vec8<A> o;
    o.set(sum);
    o.store(p.out, t * vecs + v);
  }
}

// dy[place(t, j)] = w[t, j] dout[t] and dw[t, j] = <dout[t], y[place(t, j)]>, up to kRowsAhead j
// at a time; the block's shares of their dot products are joined in a fixed order.
template <typename A>
__global__ void __launch_bounds__(512) unsort_backward_kernel(const __grid_constant__ UnsortBackwardParams q) {
  __shared__ int place[kMaxTopK];
  __shared__ float weight[kMaxTopK];
  __shared__ float part[2][16][kRowsAhead];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const UnsortParams& p = q.f;
  const size_t t = blockIdx.x;
  const int vecs = p.H / 8, n = p.T * p.k, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
  if (tid < p.k) {
    place[tid] = __ldcg(p.inv_perm + t * p.k + tid);
    weight[tid] = p.w ? __ldcg(p.w + t * p.k + tid) : 1.f;
  }
  __syncthreads();
  for (int j0 = 0, turn = 0; j0 < p.k; j0 += kRowsAhead, turn ^= 1) {
    float dot[kRowsAhead] = {};
    for (int v = tid; v < vecs; v += blockDim.x) {
      Vec8<A> d, r[kRowsAhead];
      d.load(q.d_out, t * vecs + v);
      if (q.d_w) {
#pragma unroll
        for (int j = 0; j < kRowsAhead; ++j) {
          const int row = j0 + j < p.k ? row_of(place[j0 + j], n) : -1;
          if (row >= 0) r[j].load(p.y, (size_t)row * vecs + v);
        }
      }
      float g[8];
      d.get(g);
#pragma unroll
      for (int j = 0; j < kRowsAhead; ++j) {
        if (j0 + j >= p.k) break;
        const int at = place[j0 + j], row = row_of(at, n), own = row_of(at >= 0 ? at : -1 - at, n);
        float f[8];
        if (q.d_w && row >= 0) {
          r[j].get(f);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot[j] = fmaf(g[i], f[i], dot[j]);
        }
        if (q.d_y && own >= 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = row < 0 ? 0.f : weight[j0 + j] * g[i];
          d.set(f);
          d.store(q.d_y, (size_t)own * vecs + v);
        }
      }
    }
    if (!q.d_w) continue;
    static_assert(kRowsAhead == 4, "the lanes halve four sums twice");
    // the lanes halve the sums they carry: lane l ends with the sum of j = l / 8
    const bool up = lane & 16, up2 = lane & 8;
    const float a0 = (up ? dot[2] : dot[0]) + __shfl_xor_sync(0xffffffffu, up ? dot[0] : dot[2], 16);
    const float a1 = (up ? dot[3] : dot[1]) + __shfl_xor_sync(0xffffffffu, up ? dot[1] : dot[3], 16);
    float s = (up2 ? a1 : a0) + __shfl_xor_sync(0xffffffffu, up2 ? a0 : a1, 8);
    s += __shfl_xor_sync(0xffffffffu, s, 4);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    if ((lane & 7) == 0) part[turn][warp][lane >> 3] = s;
    __syncthreads();  // (two buffers in turn: whoever writes one again is past the barrier between)
    if (tid < kRowsAhead && j0 + tid < p.k) {
      float v = part[turn][0][tid];
      for (int i = 1; i < warps; ++i) v += part[turn][i][tid];
      q.d_w[t * p.k + j0 + tid] = v;
    }
  }
}

// Many tokens: persistent blocks whose first warp brings the rows in by bulk copies, a stage of
// the ring at a time: the same columns of up to kGroupRows of a token's rows (and, backward, of
// dout).  The other warps take a stage's columns, eight a thread.  Loads by the threads
// themselves stopped at 5.6 TB/s whatever the blocks' size and number (8192 x 2 x 4096 f16:
// 35.8 to 60 us): too few of them are in flight.
constexpr int kGroupRows = 8, kRowThreads = 512, kMaxRowStages = 8;
struct RowPlan {
  int cols, chunks, groups;      // columns of a stage; column chunks of a row; groups of a token's rows
  int row_bytes, stage_bytes, stages;
};
struct RowStage {
  int place[kGroupRows];         // as in inv_perm
  float weight[kGroupRows];
};

// Sums of eight values over the warp: lane l returns that of value l / 4.
__device__ __forceinline__ float sums8(float (&v)[8]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 4, bit = 16; n >= 1; n >>= 1, bit >>= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = up ? v[i + n] : v[i], send = up ? v[i] : v[i + n];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
    }
  }
  float t = v[0];
  t += __shfl_xor_sync(0xffffffffu, t, 2);
  t += __shfl_xor_sync(0xffffffffu, t, 1);
  return t;
}

template <typename A, bool BACKWARD>
__global__ void __launch_bounds__(kRowThreads + 32, 2)
    token_rows_kernel(const __grid_constant__ UnsortBackwardParams q, const __grid_constant__ RowPlan r) {
  extern __shared__ __align__(128) uint8_t rows_smem[];
  __shared__ uint64_t full_bar[kMaxRowStages], empty_bar[kMaxRowStages];
  __shared__ RowStage info[kMaxRowStages];
  __shared__ float part[2][kRowThreads / 32][kGroupRows];
  __shared__ volatile uint32_t late;  // a taker gave up its wait: what it frees has not been filled
  const UnsortParams& p = q.f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = p.T * p.k, takers = (blockDim.x >> 5) - 1;
  const bool need_y = !BACKWARD || q.d_w;
  // a sum over a token's groups is a column's, one over the columns a row's: that runs inside
  const int outer = BACKWARD ? r.groups : r.chunks, inner = BACKWARD ? r.chunks : r.groups;
  if (threadIdx.x == 0) {
    for (int s = 0; s < r.stages; ++s) {
      ptx::mbar_init(&full_bar[s], 1);
      ptx::mbar_init(&empty_bar[s], takers);
    }
    late = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  int s = 0;
  uint32_t phase = 0;
  bool ok = true;
  auto advance = [&]() {
    if (++s == r.stages) {
      s = 0;
      phase ^= 1;
    }
  };
  if (warp == 0) {
    // ------------------------------------------------------------ the rows' copies
    auto places = [&](long long t, int& at, float& w) {
      at = -1;
      w = 0.f;
      if (t >= p.T || lane >= p.k) return;
      at = __ldcg(p.inv_perm + t * p.k + lane);
      w = p.w ? __ldcg(p.w + t * p.k + lane) : 1.f;
    };
    int at, at_next;
    float w, w_next;
    places(blockIdx.x, at_next, w_next);
    for (long long t = blockIdx.x; t < p.T && ok; t += gridDim.x) {
      at = at_next;
      w = w_next;
      places(t + gridDim.x, at_next, w_next);
      for (int o = 0; o < outer && ok; ++o)
        for (int i = 0; i < inner; ++i) {
          const int g = BACKWARD ? o : i, c = BACKWARD ? i : o, here = min(kGroupRows, p.k - g * kGroupRows), j = lane;
          const int my_at = __shfl_sync(0xffffffffu, at, (g * kGroupRows + j) & 31);
          const float my_w = __shfl_sync(0xffffffffu, w, (g * kGroupRows + j) & 31);
          const bool live = j < here && row_of(my_at, n) >= 0 && need_y;
          const int copies = __popc(__ballot_sync(0xffffffffu, live)) + (BACKWARD ? 1 : 0);
          ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(&empty_bar[s], phase ^ 1, p.wait_ns) && !late);
          if (!ok) break;
          const int col = c * r.cols, bytes = min(r.cols, p.H - col) * (int)sizeof(A);
          uint8_t* stage = rows_smem + (size_t)s * r.stage_bytes;
          if (j < here) {
            info[s].place[j] = my_at;
            info[s].weight[j] = my_w;
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_expect_tx(&full_bar[s], copies * bytes);
          __syncwarp();
          if (live)
            ptx::bulk_load(stage + (size_t)j * r.row_bytes, reinterpret_cast<const A*>(p.y) + (size_t)my_at * p.H + col, bytes,
                           &full_bar[s]);
          if (BACKWARD && lane == 31)
            ptx::bulk_load(stage + (size_t)here * r.row_bytes, reinterpret_cast<const A*>(q.d_out) + (size_t)t * p.H + col, bytes,
                           &full_bar[s]);
          advance();
        }
    }
  } else {
    // ------------------------------------------------------------ their use
    // (after a time-out they go on to the end without waiting, so that their barriers are met; no
    // stage is filled again then, as its last copies may still be under way; the places are checked
    // against the rows where they are used)
    const int v = threadIdx.x - 32;
    int turn = 0;
    for (long long t = blockIdx.x; t < p.T; t += gridDim.x)
      for (int o = 0; o < outer; ++o) {
        float sum[8] = {};  // forward: of a chunk, over the groups; backward: each row's share, over the chunks
        for (int i = 0; i < inner; ++i) {
          const int g = BACKWARD ? o : i, c = BACKWARD ? i : o, here = min(kGroupRows, p.k - g * kGroupRows);
          if (ok) {
            ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(&full_bar[s], phase, p.wait_ns));
            if (!ok && lane == 0) late = 1;  // (before the arrival below, which the producer's wait acquires)
          }
          const int col = c * r.cols + 8 * v;
          const bool on = 8 * v < r.cols && col < p.H;
          const uint8_t* stage = rows_smem + (size_t)s * r.stage_bytes;
          const RowStage& at_stage = info[s];
          if (on && !BACKWARD) {
            for (int j = 0; j < here; ++j) {
              if (row_of(at_stage.place[j], n) < 0) continue;
              Vec8<A> x;
              float f[8];
              x.load_shared(stage + (size_t)j * r.row_bytes, v);
              x.get(f);
              const float w = at_stage.weight[j];
#pragma unroll
              for (int e = 0; e < 8; ++e) sum[e] = fmaf(w, f[e], sum[e]);
            }
          }
          if (on && BACKWARD) {
            Vec8<A> x;
            float d[8];
            x.load_shared(stage + (size_t)here * r.row_bytes, v);
            x.get(d);
#pragma unroll
            for (int j = 0; j < kGroupRows; ++j) {
              if (j >= here) break;
              const int at = at_stage.place[j], row = row_of(at, n), own = row_of(at >= 0 ? at : -1 - at, n);
              float f[8];
              if (need_y && row >= 0) {
                x.load_shared(stage + (size_t)j * r.row_bytes, v);
                x.get(f);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[j] = fmaf(d[e], f[e], sum[j]);
              }
              if (q.d_y && own >= 0) {
                const float w = at_stage.weight[j];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = row < 0 ? 0.f : w * d[e];
                x.set(f);
                x.store(q.d_y, ((size_t)own * p.H + col) / 8);
              }
            }
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&empty_bar[s]);
          advance();
          if (on && !BACKWARD && i == inner - 1) {
            Vec8<A> x;
            x.set(sum);
            x.store(p.out, ((size_t)t * p.H + col) / 8);
          }
        }
        if (BACKWARD && q.d_w) {
          const int here = min(kGroupRows, p.k - o * kGroupRows);
          const float mine = sums8(sum);
          if ((lane & 3) == 0) part[turn][warp - 1][lane >> 2] = mine;
          asm volatile("bar.sync 1, %0;" ::"r"(32 * takers) : "memory");
          if (v < here) {
            float total = part[turn][0][v];
            for (int e = 1; e < takers; ++e) total += part[turn][e][v];
            q.d_w[t * p.k + o * kGroupRows + v] = total;
          }
          turn ^= 1;  // (whoever writes a buffer again is past the barrier between)
        }
      }
  }
  if (!ok && lane == 0) {
    // a copy waited for in vain may still land: report, and stay until it surely has
    report_status(&g_sort_status, kStatusTimeoutMain);
    const uint64_t since = ptx::globaltimer_ns();
    while (ptx::globaltimer_ns() - since < kLandingNs) __nanosleep(1000);
  }
}

// The gradient of the top-k weights into the logits, a warp per token.  With S = sum_i w_i g_i:
//   softmax over the k selected   dl_j = w_j (g_j - S)
//   sigmoids over their sum       dl_j = w_j (1 - sigmoid(l_j)) (g_j - S)
//   softmax over all E            dl_e = p_e (g_e - S), g_e = 0 where e was not selected
// added where an expert was selected twice, in the order of j; 0 elsewhere.  A term whose g is 0
// adds nothing to S whatever its weight, and a token all of whose g are 0 gets zeros: one that a mask
// leaves no expert has NaN weights, and the zero gradients of its dropped assignments stay zeros.
__global__ void __launch_bounds__(256) route_backward_kernel(const __grid_constant__ RouteBackwardParams p) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const size_t t = (size_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= (size_t)p.T) return;
  const float* logits = p.logits + t * p.E;
  const bool all = p.gating == kGatingSoftmaxAll;
  float top = -INFINITY, sum = 0.f, l[kMaxExperts / 32];
  if (all) {
#pragma unroll
    for (int i = 0; i < kMaxExperts / 32; ++i)
      if (32 * i < p.E) l[i] = lane + 32 * i < p.E ? __ldcg(logits + lane + 32 * i) : -INFINITY;
  }
  int e = -1;
  float g = 0.f, w = 0.f;
  if (lane < p.k) {
    e = __ldcg(p.idx + t * p.k + lane);
    if (e >= p.E) e = -1;
    g = __ldcg(p.d_w + t * p.k + lane);
    w = __ldcg(p.w + t * p.k + lane);
  }
  float s = g == 0.f ? 0.f : w * g;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  float* out = p.d_logits + t * p.E;
  const bool none = __all_sync(0xffffffffu, g == 0.f);
  float part = all ? g : w * (g - s);
  if (p.gating == kGatingSigmoid && e >= 0) part *= 1.f / (1.f + expf(__ldcg(logits + e)));
  if (none) part = 0.f;
  if (all) {
#pragma unroll
    for (int i = 0; i < kMaxExperts / 32; ++i)
      if (32 * i < p.E) top = fmaxf(top, l[i]);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
#pragma unroll
    for (int i = 0; i < kMaxExperts / 32; ++i) {
      if (32 * i >= p.E) break;  // (every expert slot for 8 experts: 6.3 us for 8192 tokens)
      l[i] = lane + 32 * i < p.E && !none ? expf(l[i] - top) : 0.f;
      sum += l[i];
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (none) sum = 1.f;
  }
#pragma unroll
  for (int i = 0; i < kMaxExperts / 32; ++i) {
    if (32 * i >= p.E) break;
    const int c = lane + 32 * i;
    float v = 0.f;
    for (int j = 0; j < p.k; ++j) {
      const float add = __shfl_sync(0xffffffffu, part, j);
      if (__shfl_sync(0xffffffffu, e, j) == c) v += add;
    }
    if (all) v = l[i] / sum * (v - s);
    if (c < p.E) out[c] = v;
  }
}

// Threads of a block that takes one token.
int token_threads(int H) { return min(512, ceil_div(H / 8, 32) * 32); }

// The ring of the persistent blocks: stages of at most 48 KB, of at least two per block.
constexpr int kRowSmem = 222 * 1024, kRowOther = 3 * 1024, kMaxStage = 48 * 1024;  // (other: what else a block takes)
template <typename A, bool BACKWARD>
cudaError_t launch_rows(const UnsortBackwardParams& q, cudaStream_t stream, bool& taken) {
  const int H = q.f.H, k = q.f.k, rows = min(k, kGroupRows) + (BACKWARD ? 1 : 0);
  const int most = min(8 * kRowThreads, kMaxStage / (rows * (int)sizeof(A)) / 8 * 8);
  RowPlan r{};
  r.chunks = ceil_div(H, most);
  r.cols = ceil_div(H / 8, r.chunks) * 8;
  r.groups = ceil_div(k, kGroupRows);
  r.row_bytes = r.cols * (int)sizeof(A);
  r.stage_bytes = rows * r.row_bytes;
  const int threads = ceil_div(r.cols / 8, 32) * 32 + 32;
  const int per_sm = max(1, min(min(16, 2 * (kRowThreads + 32) / threads), kRowSmem / (2 * r.stage_bytes + kRowOther)));
  r.stages = min(kMaxRowStages, (kRowSmem / per_sm - kRowOther) / r.stage_bytes);
  const int blocks = per_sm * device_sms();
  // (fewer tokens are done sooner by a block each: forward 608 x 4 x 2880 4.4 us against 5.0, 1824 x 4
  // 9.9 against 10.1, 4096 x 4 21.7 against 20.1; backward 304 x 4 4.4 against 5.0, 608 x 4 7.7 against
  // 7.4, 1216 x 2 x 4096 12.9 against 10.4)
  taken = q.f.T >= (BACKWARD ? 3 : 6) * blocks;
  if (!taken) return cudaSuccess;
  auto kern = token_rows_kernel<A, BACKWARD>;
  static SmemOptIn opt_in;
  const cudaError_t e = opt_in.ensure(kern, kRowSmem);
  return e != cudaSuccess ? e : launch_pdl(kern, dim3(blocks), dim3(threads), r.stages * r.stage_bytes, stream, q, r);
}

template <typename A>
cudaError_t unsort_t(const UnsortParams& p, cudaStream_t stream) {
  UnsortBackwardParams q{};
  q.f = p;
  bool taken = false;
  const cudaError_t e = launch_rows<A, false>(q, stream, taken);
  return taken || e != cudaSuccess ? e : launch_pdl(unsort_kernel<A>, dim3(p.T), dim3(token_threads(p.H)), 0, stream, p);
}
template <typename A>
cudaError_t unsort_backward_t(const UnsortBackwardParams& q, cudaStream_t stream) {
  bool taken = false;
  const cudaError_t e = launch_rows<A, true>(q, stream, taken);
  return taken || e != cudaSuccess ? e
                                   : launch_pdl(unsort_backward_kernel<A>, dim3(q.f.T), dim3(token_threads(q.f.H)), 0, stream, q);
}

}  // namespace

uint32_t* sort_status_word() {
  void* p = nullptr;
  return cudaGetSymbolAddress(&p, g_sort_status) == cudaSuccess ? static_cast<uint32_t*>(p) : nullptr;
}

cudaError_t launch_sort(const SortParams& p, cudaStream_t stream) {
  if ((long long)p.T * p.k <= kFewAssignments) return launch_pdl(sort_few_kernel, dim3(p.T + 1), dim3(kFewThreads), 0, stream, p);
  cudaError_t e = launch_pdl(order_kernel, dim3(kOrderBlocks), dim3(kOrderThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  // warps of a block: as many as leave four blocks per SM, and as many blocks as reside
  constexpr int kSmem = 224 * 1024;
  const int ring = kGatherStages * p.row_bytes;
  const int warps = max(1, min(4, kSmem / 4 / ring)), per_sm = max(1, min(16, kSmem / (warps * ring + 1024)));
  static SmemOptIn opt_in;
  e = opt_in.ensure(gather_kernel, kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(gather_kernel, dim3(min(ceil_div(p.T, warps), per_sm * device_sms())), dim3(32 * warps), warps * ring, stream, p);
}

cudaError_t launch_unsort(const UnsortParams& p, int dtype, cudaStream_t stream) {
  return dtype == kDtypeBf16  ? unsort_t<__nv_bfloat16>(p, stream)
         : dtype == kDtypeF16 ? unsort_t<__half>(p, stream)
                              : unsort_t<float>(p, stream);
}

cudaError_t launch_unsort_backward(const UnsortBackwardParams& q, int dtype, cudaStream_t stream) {
  return dtype == kDtypeBf16  ? unsort_backward_t<__nv_bfloat16>(q, stream)
         : dtype == kDtypeF16 ? unsort_backward_t<__half>(q, stream)
                              : unsort_backward_t<float>(q, stream);
}

cudaError_t launch_route_backward(const RouteBackwardParams& p, cudaStream_t stream) {
  return launch_pdl(route_backward_kernel, dim3(ceil_div(p.T, 8)), dim3(256), 0, stream, p);
}

}  // namespace moe
