// Page tables, sequence lengths and slot maps of a serving step, built on the GPU from the
// requests' lengths.
//
// With P = 128 tokens per page, request b holds held_b = ceil(prev_b / P) pages and needs
// need_b = ceil((prev_b + new_b) / P) - held_b more. They are taken from the free list in
// request order, so the whole assignment follows from two exclusive prefix sums over the batch:
// cu_b (new tokens before request b) and first_b (fresh pages before it). Token t of request b
// sits at position prev_b + t - cu_b, and its page is either one the request held or entry
// first_b + (block - held_b) of the free list: no part of the answer waits for another part's
// store, so one launch does everything.
//
// Every CTA computes both scans itself (B is at most kMaxRequests; the loads come from L2) and
// keeps them in shared memory, then finds the request of a token or of a fresh page by binary
// search there. The bytes are few (a 32768-token step writes 0.5 MB): the launch and the chain
// load -> scan -> search -> page -> store bound the time, so a step of few tokens takes one CTA.
// Measured, replayed from a graph: 2.5 us for 8 requests of one token, 4.1 us for 61 requests and
// 65453 token rows (128 GB/s), 6.6 us for 512 requests behind 256 shared pages (262656 token rows and
// 131072 shared entries, 2.6 MB: 0.4 TB/s). A launch that is one load and one store deep takes 1.9 us.
#include "common.cuh"
#include "host_util.h"
#include "kernels.h"

MSA_DEFINE_ERROR_WORD(tables)

namespace msa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Lens {
  int32_t prev, fresh_tok;  // clamped to the table's extent
  bool bad;
};

__device__ __forceinline__ Lens read_lens(const PageTablesArgs& a, int b) {
  const int64_t cap = (int64_t)a.max_blocks * MSA_BLOCK_TOKENS;
  const int32_t p0 = a.prev_lens[b], n0 = a.new_lens[b];
  const int64_t p = p0 < 0 ? 0 : (p0 > cap ? cap : p0);
  const int64_t n = n0 < 0 ? 0 : (n0 > cap - p ? cap - p : n0);
  return {(int32_t)p, (int32_t)n, p != p0 || n != n0};
}
__device__ __forceinline__ int32_t pages_of(int32_t tokens) {
  return tokens / MSA_BLOCK_TOKENS + (tokens % MSA_BLOCK_TOKENS != 0);
}

// Largest i in [0, n) with v[i] <= x (v ascending, v[0] <= x).
__device__ __forceinline__ int last_not_above(const int32_t* v, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) page_tables_kernel(const PageTablesArgs a) {
  extern __shared__ int32_t s_scan[];  // cu [B + 1], first [B + 1]
  __shared__ int64_t w_tok[kWarps];
  __shared__ int32_t w_page[kWarps];
  int32_t* cu = s_scan;
  int32_t* first = s_scan + a.B + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  // ---------------- the two scans; token sums in 64 bits, kept saturated at INT32_MAX
  int64_t tok = 0;
  int32_t pages = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const Lens l = read_lens(a, b);
    bad |= l.bad;
    tok += l.fresh_tok;
    pages += pages_of(l.prev + l.fresh_tok) - pages_of(l.prev);
  }
  int64_t ti = tok;
  int32_t pi = pages;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t2 = __shfl_up_sync(0xffffffffu, ti, o);
    const int32_t p2 = __shfl_up_sync(0xffffffffu, pi, o);
    if (lane >= o) {
      ti += t2;
      pi += p2;
    }
  }
  if (lane == 31) {
    w_tok[warp] = ti;
    w_page[warp] = pi;
  }
  __syncthreads();
  int64_t tbase = ti - tok, ttotal = 0;
  int32_t pbase = pi - pages, ptotal = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) {
      tbase += w_tok[w];
      pbase += w_page[w];
    }
    ttotal += w_tok[w];
    ptotal += w_page[w];
  }
  const int32_t used_in = a.pages_used[0];
  const int32_t used = used_in < 0 ? 0 : (used_in > a.num_free ? a.num_free : used_in);
  const int32_t avail = a.num_free - used;
  const bool lead = blockIdx.x == 0;
  for (int b = b0; b < b1; ++b) {
    const Lens l = read_lens(a, b);
    const int32_t held = pages_of(l.prev), need = pages_of(l.prev + l.fresh_tok) - held;
    const int32_t c = (int32_t)min(tbase, (int64_t)INT32_MAX);
    cu[b] = c;
    first[b] = pbase;
    if (lead) {
      a.cu_tokens[b] = c;
      // a request that the free list cannot serve whole keeps the tokens its pages hold
      int64_t s = l.prev + l.fresh_tok;
      if (pbase + need > avail) {
        const int64_t got = held + (int64_t)max(0, avail - pbase);
        s = min(s, got * MSA_BLOCK_TOKENS);
      }
      a.seq_lens[b] = (int32_t)s;
    }
    tbase += l.fresh_tok;
    pbase += need;
  }
  const int32_t total = (int32_t)min(ttotal, (int64_t)INT32_MAX);
  if (tid == 0) {
    cu[a.B] = total;
    first[a.B] = ptotal;
    if (lead) {
      a.cu_tokens[a.B] = total;
      a.pages_used_out[0] = used + min(ptotal, avail);
      uint32_t e = 0;
      if (ptotal > avail) e |= kErrNoPage;
      if (ttotal > a.T || used != used_in) e |= kErrBadBlock;
      if (e) msa_record_error(e);
    }
  }
  if (lead && bad) msa_record_error(kErrBadBlock);
  __syncthreads();
  const int64_t gtid = (int64_t)blockIdx.x * kThreads + tid;
  const int64_t gthreads = (int64_t)gridDim.x * kThreads;
  // ---------------- slots and positions of the token rows
  for (int64_t t = gtid; t < a.T; t += gthreads) {
    int32_t slot = -1, pos = -1;
    if (t < total) {
      const int b = last_not_above(cu, a.B, (int32_t)t);
      const Lens l = read_lens(a, b);
      pos = l.prev + ((int32_t)t - cu[b]);
      const int32_t blk = pos / MSA_BLOCK_TOKENS, held = pages_of(l.prev);
      int32_t page = -1;
      bool have = true;
      if (blk < held) {
        page = a.page_table[(int64_t)b * a.max_blocks + blk];
      } else {
        const int32_t at = first[b] + blk - held;
        have = at < avail;
        if (have) page = a.free_pages[used + at];
      }
      if (have) {
        if (page >= 0 && page < a.num_pages) slot = page * MSA_BLOCK_TOKENS + pos % MSA_BLOCK_TOKENS;
        else msa_record_error(kErrBadPage);
      }
    }
    a.slot_map[t] = slot;
    a.positions[t] = pos;
  }
  // ---------------- table entries of the fresh pages
  for (int64_t i = gtid; i < ptotal; i += gthreads) {
    const int b = last_not_above(first, a.B, (int32_t)i);
    const int32_t held = pages_of(read_lens(a, b).prev);
    int32_t page = -1;
    if (i < avail) {
      page = a.free_pages[used + i];
      if (page < 0 || page >= a.num_pages) {
        page = -1;
        msa_record_error(kErrBadPage);
      }
    }
    a.page_table[(int64_t)b * a.max_blocks + held + ((int32_t)i - first[b])] = page;
  }
  // ---------------- the shared prefix's entries, for every request that holds all of it
  if (a.num_shared > 0) {
    const int64_t gwarps = (int64_t)gridDim.x * kWarps;
    for (int64_t b = (int64_t)blockIdx.x * kWarps + warp; b < a.B; b += gwarps) {
      if ((int64_t)read_lens(a, (int)b).prev < (int64_t)a.num_shared * MSA_BLOCK_TOKENS) continue;
      for (int j = lane; j < a.num_shared; j += 32) {
        int32_t page = a.shared_pages[j];
        if (page < 0 || page >= a.num_pages) {
          page = -1;
          msa_record_error(kErrBadPage);
        }
        a.page_table[b * a.max_blocks + j] = page;
      }
    }
  }
}

}  // namespace

cudaError_t launch_page_tables(const PageTablesArgs& a, cudaStream_t stream) {
  // about four token rows or sixteen shared entries per thread, at most two CTAs per SM
  const int64_t rows = (int64_t)a.T / 4 + (int64_t)a.B * a.num_shared / 16;
  int64_t grid = (rows + kThreads - 1) / kThreads;
  const int64_t cap = 2 * (int64_t)sm_count();
  grid = grid < 1 ? 1 : (grid > cap ? cap : grid);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)2 * (a.B + 1) * sizeof(int32_t);
  cfg.stream = stream;
  // the limit of the largest batch for all of them: were it the call's own, one thread could lower it
  // between another's raise and launch
  constexpr size_t kMaxSmem = (size_t)2 * (kMaxRequests + 1) * sizeof(int32_t);
  static std::atomic<size_t> raised[kMaxDevices];
  return launch_with_smem(page_tables_kernel, kMaxSmem, raised,
                          [&] { return cudaLaunchKernelEx(&cfg, page_tables_kernel, a); });
}

}  // namespace msa
