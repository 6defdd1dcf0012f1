// The plan of a batch (include/q4_serve.h): offsets, positions, slots and pages of the new
// tokens from the requests' lengths.
//
// With n_s new tokens behind len_s (0 where the sequence is reset), P tokens a page:
//   have_s = ceil(len_s / P), need_s = ceil((len_s + n_s) / P) - have_s,
//   q_offsets = exclusive sum of n, page j of the sequence's new ones is number
//   (exclusive sum of need)_s + j from the top of the stack.
// Two scans over the sequences (three with pages given back), then every row finds its
// sequence by bisection of the offsets and writes its position and slot; the row at a new
// page's first token enters the page in the block table. Nothing is carried from workgroup
// to workgroup but the scans' results, so a plan is one launch where one workgroup is enough
// for the rows, and two otherwise.
//
// What bounds it is latency: 48 sequences of one token read and write 1.2 KB and take 4.2 us in a graph, a chain of
// lengths, two scans, page and slot; one sequence takes 3.7. The scans go through DPP and pages
// given back are copied by a wavefront a sequence (61 prompts of 4001 tokens, a fifth of their places
// reused: 16.2 -> 11.9 us), by no more threads than the sequences need (10.7).
#include "q4_device.h"
#include "q4_internal.h"

namespace q4 {
namespace {

// Exclusive sums over the workgroup of two 64-bit numbers a thread, and the totals. Each call has its own LDS.
struct Pair64 {
  int64_t a, b;
};
template <int CTRL, int ROWS>
__device__ __forceinline__ int64_t plus_dpp(int64_t v) {
  const int lo = __builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(v >> 32), CTRL, ROWS, 0xF, false);
  return v + (int64_t)((uint64_t)(uint32_t)hi << 32 | (uint32_t)lo);
}
__device__ __forceinline__ int64_t wave_scan(int64_t v) {  // inclusive: rows of 16 lanes, then from row to row
  v = plus_dpp<0x111, 0xF>(v);
  v = plus_dpp<0x112, 0xF>(v);
  v = plus_dpp<0x114, 0xF>(v);
  v = plus_dpp<0x118, 0xF>(v);
  v = plus_dpp<0x142, 0xA>(v);
  return plus_dpp<0x143, 0xC>(v);
}
__device__ __forceinline__ Pair64 block_scan(Pair64 v, Pair64* wave_sums, Pair64* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = (int)(blockDim.x >> 6);
  const Pair64 incl{wave_scan(v.a), wave_scan(v.b)};
  if (lane == kWave - 1) wave_sums[wave] = incl;
  __syncthreads();
  Pair64 before{0, 0}, all{0, 0};
  for (int w = 0; w < waves; ++w) {
    const Pair64 s = wave_sums[w];
    if (w < wave) before.a += s.a, before.b += s.b;
    all.a += s.a, all.b += s.b;
  }
  *total = all;
  return Pair64{before.a + incl.a - v.a, before.b + incl.b - v.b};
}

// What a row needs of its sequence.
struct PlanSeq {
  int len, first_page;  // tokens before the new ones; place of its first new page from the stack's top
};

// `seqs` offsets behind `first`: off(i) is q_offsets[i]. The row's position in its sequence's slot.
template <typename Off, typename Seq>
__device__ __forceinline__ void plan_row(const PlanArgs& a, int row, int total, int avail, Off off, Seq seq) {
  int slot = -1, position = 0;
  if (row < total) {
    int lo = 0, hi = a.seqs;  // off(lo) <= row < off(hi)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (off(mid) <= row) lo = mid; else hi = mid;
    }
    const PlanSeq s = seq(lo);
    const int t = s.len + row - off(lo);
    const int block = t / a.page_size, in_page = t - block * a.page_size;
    const int have = (s.len + a.page_size - 1) / a.page_size;
    int page = -1;
    if (block < a.max_blocks) {
      int32_t* entry = a.block_table + (int64_t)lo * a.max_blocks + block;
      if (block < have || !a.free_pages) {
        page = *entry;
      } else if (s.first_page + (block - have) < avail) {
        page = a.free_pages[avail - 1 - (s.first_page + (block - have))];
        if (in_page == 0) *entry = page;
      }
    }
    if ((unsigned)page < (unsigned)a.pages) slot = page * a.page_size + in_page;
    position = (int)((uint32_t)(a.starts ? a.starts[lo] : 0) + (uint32_t)t);
  }
  a.positions[row] = position;
  a.slots[row] = slot;
}

// One workgroup: the scans, the pages given back, all results a sequence has; with FILL the
// rows too (seqs <= kPlanThreads), else what the rows need is left in the workspace.
template <bool FILL>
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(PlanArgs a) {
  __shared__ Pair64 wave_sums[2][kPlanThreads / kWave];
  __shared__ int2 given[kPlanThreads];  // pages that a sequence gives back, and where to
  __shared__ int off_of[FILL ? kPlanThreads + 1 : 1];
  __shared__ PlanSeq seq_of[FILL ? kPlanThreads : 1];
  const int lane = threadIdx.x & 63;
  const int threads = (int)blockDim.x;
  const int page = a.page_size;
  const int cap = a.max_blocks * page;
  int64_t avail = a.free_pages ? min(max(a.free_count[0], 0), a.pages) : 0;

  // pages of the sequences that are reset
  if (a.reset && a.free_pages) {
    for (int base = 0; base < a.seqs; base += threads) {
      const int s = base + (int)threadIdx.x;
      int n = 0;
      if (s < a.seqs && a.reset[s] != 0) n = (min(max(a.kv_lens[s], 0), cap) + page - 1) / page;
      Pair64 total;
      const int64_t at = avail + block_scan(Pair64{n, 0}, wave_sums[0], &total).a;
      if (total.a > 0) {
        given[threadIdx.x] = make_int2(n, (int)(at < a.pages ? at : a.pages));
        __syncthreads();
        for (int i = (int)threadIdx.x >> 6; i < threads && base + i < a.seqs; i += threads >> 6) {  // a wavefront a sequence
          const int2 g = given[i];
          const int32_t* from = a.block_table + (int64_t)(base + i) * a.max_blocks;
          for (int j = lane; j < g.x; j += kWave)
            if (j < a.pages - g.y) a.free_pages[g.y + j] = from[j];
        }
      }
      __syncthreads();  // given and wave_sums may be written again
      avail += total.a;
    }
    avail = avail < a.pages ? avail : a.pages;
    __syncthreads();  // the stack is complete before pages are taken from it
  }

  int64_t rows = 0, taken = 0, wanted = 0;
  for (int base = 0; base < a.seqs; base += threads) {
    const int s = base + (int)threadIdx.x;
    const bool there = s < a.seqs;
    int len = 0, fresh = 0;
    if (there) {
      len = a.reset && a.reset[s] != 0 ? 0 : min(max(a.kv_lens[s], 0), cap);
      fresh = a.new_lens ? min(max(a.new_lens[s], 0), a.tokens) : 1;
    }
    Pair64 total;
    const int64_t first = rows + block_scan(Pair64{there ? fresh : 0, 0}, wave_sums[0], &total).a;
    const int off = (int)(first < a.tokens ? first : a.tokens);
    const int end = (int)(first + fresh < a.tokens ? first + fresh : a.tokens);
    rows += total.a;
    const int have = (len + page - 1) / page;
    const int want = there ? (int)(((int64_t)len + (end - off) + page - 1) / page) : have;
    const int need = min(want, a.max_blocks) - have;  // have <= max_blocks
    const Pair64 ex = block_scan(Pair64{need, want - have}, wave_sums[1], &total);
    const int64_t place = taken + ex.a;
    taken += total.a;
    wanted += total.b;
    int granted = need;
    if (a.free_pages) granted = (int)(avail - place < 0 ? 0 : avail - place < need ? avail - place : need);
    if (there) {
      const int64_t room = (int64_t)(have + granted) * page, full = (int64_t)len + (end - off);
      const PlanSeq mine{len, (int)place};
      a.q_offsets[s] = off;
      a.kv_lens_out[s] = (int)(full < room ? full : room);
      if (FILL) {
        off_of[s] = off;
        seq_of[s] = mine;
      } else {
        *reinterpret_cast<int2*>(a.seq_info + 2 * s) = make_int2(mine.len, mine.first_page);
      }
    }
  }
  // pages go out in order until there are none
  const int64_t granted_all = a.free_pages && avail < taken ? avail : taken, lacking = wanted - granted_all;
  const int total_rows = (int)(rows < a.tokens ? rows : a.tokens);
  if (threadIdx.x == 0) {
    a.q_offsets[a.seqs] = total_rows;
    a.lacking[0] = (int)(lacking < 0x7FFFFFFF ? lacking : 0x7FFFFFFF);
    if (a.free_pages) a.free_count_out[0] = (int)(avail - granted_all);
    if (!FILL) a.seq_info[2 * a.seqs] = (int)avail;
  }
  if (FILL) {
    __syncthreads();
    for (int row = (int)threadIdx.x; row < a.tokens; row += threads)
      plan_row(a, row, total_rows, (int)avail, [&](int i) { return off_of[i]; }, [&](int i) { return seq_of[i]; });
  }
}

__global__ __launch_bounds__(256) void plan_rows_kernel(PlanArgs a) {
  const int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (row >= a.tokens) return;
  const int2* info = reinterpret_cast<const int2*>(a.seq_info);
  plan_row(a, (int)row, a.q_offsets[a.seqs], a.seq_info[2 * a.seqs], [&](int i) { return a.q_offsets[i]; },
           [&](int i) {
             const int2 v = info[i];
             return PlanSeq{v.x, v.y};
           });
}

}  // namespace

hipError_t launch_plan(const PlanArgs& a, hipStream_t stream) {
  const int threads = a.seqs <= kPlanSmall ? kPlanSmall : kPlanThreads;
  if (plan_one_launch(a.seqs, a.tokens)) {
    hipLaunchKernelGGL((plan_kernel<true>), dim3(1), dim3(threads), 0, stream, a);
  } else {
    hipLaunchKernelGGL((plan_kernel<false>), dim3(1), dim3(threads), 0, stream, a);
    if (a.tokens > 0)
      hipLaunchKernelGGL(plan_rows_kernel, dim3((unsigned)((a.tokens + 255) / 256)), dim3(256), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace q4
