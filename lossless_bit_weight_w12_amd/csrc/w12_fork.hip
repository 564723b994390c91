// Pages that requests share: block tables brought in line where a request continues another
// one (w12_kv_fork), the copies and moves of pages in the caches (w12_kv_copy), and a range of
// the pool cleared of pages (w12_kv_compact).
//
// The counts of holders lie in refs [n_pages]; behind them the calls' own words: per page the
// change of its count and the mark of a call under way (both zero between calls), per page a
// rank and a target of w12_kv_compact, and the workgroups' counts.
#include "w12.h"
#include "w12_fork.h"
#include "w12_plan.h"

namespace w12 {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kForkWG = 256;        // workgroups of a launch, at most (one count each)
constexpr uint32_t kEntries = 8192;      // table entries of a workgroup in LDS at a time
constexpr uint32_t kWriter = 0x10000u;   // a mark of a request that writes

// x / d, for x d < 2^32: inv = floor((2^32 - 1) / d) is less than 2^32 / d by 1 at most, the product by less
// than x / 2^32 + 1, so the quotient is it or one more.
__device__ __forceinline__ uint32_t divide(uint32_t x, uint32_t d, uint32_t inv) {
  const uint32_t q = __umulhi(x, inv);
  return q + (x - q * d >= d);
}

// Words that one workgroup alone uses in a launch.
__device__ __forceinline__ int32_t load_here(const int32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}
__device__ __forceinline__ void add_here(int32_t* p, int32_t v) {
  __hip_atomic_fetch_add(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}
__device__ __forceinline__ void max_here(int32_t* p, int32_t v) {
  __hip_atomic_fetch_max(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}

// Sum over the workgroup's threads, the same in all of them.
template <int T>
__device__ __forceinline__ uint32_t block_sum(uint32_t v, uint32_t* s_w) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s_w[threadIdx.x >> 6] = v;
  __syncthreads();
  uint32_t all = 0;
#pragma unroll
  for (int w = 0; w < T / 64; ++w) all += s_w[w];
  return all;
}

// Number of set flags in threads before this one, and in all of them.
template <int T>
__device__ __forceinline__ uint32_t block_rank(bool flag, uint32_t* s_w, uint32_t& all) {
  const uint64_t b = __ballot(flag);
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __syncthreads();
  if (lane == 0) s_w[wave] = (uint32_t)__popcll(b);
  __syncthreads();
  uint32_t before = (uint32_t)__popcll(b & ((1ull << lane) - 1ull));
  all = 0;
#pragma unroll
  for (int w = 0; w < T / 64; ++w) {
    if (w < (int)wave) before += s_w[w];
    all += s_w[w];
  }
  return before;
}

// One request of w12_kv_fork: what it shall hold.
struct Fork {
  int32_t src;           // row that it continues, -1: none
  uint32_t held, keep;   // pages of its row now, pages of src that it takes
  uint32_t want;         // pages afterwards
  int32_t len;
  uint32_t off, rows;
  bool writes;           // it adds rows to the last page it takes
  bool served;
};

__device__ __forceinline__ Fork fork_req(const ForkArgs& a, uint32_t r, bool& bad) {
  Fork f;
  const int32_t lo = a.req_off[r], hi = a.req_off[r + 1], len = a.len[r], own = a.held[r];
  const int32_t src = a.parent ? a.parent[r] : (int32_t)r;
  bad |= lo < 0 || hi < lo || hi > (int32_t)a.m;
  const bool whole = own >= 0 && (uint32_t)own <= a.max_pages;
  const bool known = src >= 0 && (uint32_t)src < a.max_req;
  const int32_t have = known ? a.held[src] : 0;
  const uint32_t page = 1u << a.page_shift, rows = (uint32_t)(hi - lo);
  f.off = (uint32_t)lo;
  f.rows = rows;
  f.len = len;
  f.held = whole ? (uint32_t)own : 0u;
  f.served = whole && len >= 0 && (known ? have >= 0 && (uint32_t)have <= a.max_pages : src == -1) &&
             (int64_t)len + rows <= (int64_t)a.max_pages << a.page_shift &&
             ((uint64_t)(uint32_t)len + page - 1) >> a.page_shift <= (uint64_t)(uint32_t)have;
  if (f.served) {
    f.src = src;
    f.keep = ((uint32_t)len + page - 1) >> a.page_shift;
    f.want = (uint32_t)(((uint64_t)len + rows + page - 1) >> a.page_shift);
    f.writes = ((uint32_t)len & (page - 1)) != 0 && rows > 0;
  } else {   // it keeps what it holds
    f.src = (int32_t)r;
    f.keep = f.want = f.held;
    f.writes = false;
  }
  return f;
}

// The requests in LDS.  Flags of keep: the request writes into the last page it takes, and gets a
// copy of it.
constexpr uint32_t kWrites = 1u << 31, kCopied = 1u << 30, kKeep = kCopied - 1u;
template <int T, int N>
struct ForkLds {
  int32_t src[N], len[N];   // len: -1: not served
  uint32_t held[N], keep[N], need[N + 1], off[N + 1];
  int32_t old[kEntries];
  uint32_t w[T / 64], cols, sum[2], last;
};

// Reads them, a thread some in a row; need[r + 1]: pages behind those it takes.  Whether the offsets
// are none; T * ceil(N / T) requests at most.
template <int T, int N>
__device__ __forceinline__ bool fork_requests(const ForkArgs& a, ForkLds<T, N>& s) {
  const uint32_t t = threadIdx.x, n = a.n_req, per = (n + T - 1) / T;
  if (t == 0) s.cols = s.need[0] = 0;
  __syncthreads();
  uint32_t cols = 0;
  bool bad = false;
#pragma unroll
  for (uint32_t i = 0; i < N / T; ++i) {
    const uint32_t r = t * per + i;
    if (i >= per || r >= n) break;
    const Fork f = fork_req(a, r, bad);
    s.src[r] = f.src;
    s.held[r] = f.held;
    s.keep[r] = f.keep | (f.writes ? kWrites : 0u);
    s.need[r + 1] = f.want - f.keep;
    s.len[r] = f.served ? f.len : -1;
    s.off[r] = f.off;
    if (r + 1 == n) s.off[n] = f.off + f.rows;
    cols = max(cols, max(f.held, f.keep));
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) cols = max(cols, (uint32_t)__shfl_xor((int)cols, o));
  if ((t & 63) == 0) atomicMax(&s.cols, cols);
  return __syncthreads_or(bad);
}

// The table's columns c0 .. c0 + w - 1 as they are.
template <int T, int N>
__device__ __forceinline__ void fork_columns(const ForkArgs& a, ForkLds<T, N>& s, uint32_t c0, uint32_t w) {
  __syncthreads();
  const uint32_t inv = 0xffffffffu / w;
  for (uint32_t e = threadIdx.x; e < w * a.n_req; e += T) {
    const uint32_t r = divide(e, w, inv), j = e - r * w;
    s.old[j * a.n_req + r] = c0 + j < s.held[r] ? a.table[(uint64_t)r * a.max_pages + c0 + j] : -1;
  }
  __syncthreads();
}

// What request r's place in column c holds (x) and will hold of src's pages (y), -1: nothing.
template <int T, int N>
__device__ __forceinline__ void entry(const ForkArgs& a, const ForkLds<T, N>& s, uint32_t r, uint32_t j, uint32_t c,
                                      int32_t& x, int32_t& y, bool& tail) {
  const uint32_t n = a.n_req, flags = s.keep[r], keep = flags & kKeep;
  x = s.old[j * n + r];
  y = -1;
  tail = false;
  if (c < keep) {
    const int32_t src = s.src[r];
    y = (uint32_t)src < n ? s.old[j * n + (uint32_t)src] : a.table[(uint64_t)(uint32_t)src * a.max_pages + c];
    tail = c + 1 == keep && (flags & kWrites);
  }
}

// The columns that somebody holds are dealt to the workgroups, of both halves of w12_kv_fork alike:
// the holders of a page hold it in the same column (a request that continues another one has its
// first tokens in the same places), so one workgroup sees everything about a page, and what it
// counts per page needs no wider scope than its own.  A column's old entries are in LDS, so that
// the rows can change places.  The first half counts: the change of each page's holders, the
// requests that write into their last page (the lowest may keep it if nobody else holds it), and
// the pages nobody holds any longer; the second knows from the sums where the pages it gives back
// go and whether there are enough, and writes.  Entries that stay are passed over before any
// atomic, so a prompt's shared pages cost nothing.
//
// Two launches, or one where a single workgroup takes all columns.  Bound by latency (dependent
// reads behind the launches): 4 requests 8.5 us in one launch, 96 of 515 places 16 us in two (with the
// counts per page at the device's scope, that is past the L2, a third more).
struct Columns {   // of a workgroup, and how many of them are in LDS at a time
  uint32_t begin, end, width;
};
template <int T, int N>
__device__ __forceinline__ Columns columns(const ForkArgs& a, const ForkLds<T, N>& s) {
  const uint32_t per = a.grid == 1 ? s.cols : (s.cols + a.grid - 1) / a.grid;
  return Columns{blockIdx.x * per, min(s.cols, (blockIdx.x + 1) * per), max(1u, min(per, a.at_once))};
}

// A page in the middle of a call: its mark, and who will hold it but for those that write into it (read
// together: one read less to wait for).
struct Page {
  int32_t mark, holders;
};
__device__ __forceinline__ Page page_now(const ForkArgs& a, int32_t p) {
  const int32_t change = load_here(a.refs + a.n_pages + p), mark = load_here(a.refs + 2ull * a.n_pages + p);
  return Page{mark, a.refs[p] + change};
}

// The first half: the number of pages that this workgroup's columns give back.
template <int T, int N>
__device__ __forceinline__ uint32_t fork_look(const ForkArgs& a, ForkLds<T, N>& s) {
  const uint32_t t = threadIdx.x, n = a.n_req;
  int32_t* const delta = a.refs + a.n_pages;
  int32_t* const mark = delta + a.n_pages;
  uint32_t freed = 0;
  auto valid = [&](int32_t p) { return (uint32_t)p < a.n_pages; };
  auto page = [&](int32_t p, bool read) { return read ? page_now(a, p) : Page{0, 0}; };
  const Columns k = columns(a, s);
  for (uint32_t c0 = k.begin; c0 < k.end; c0 += k.width) {
    const uint32_t w = min(k.width, k.end - c0), all = w * n;
    fork_columns(a, s, c0, w);
    bool any = false;
    for (uint32_t e = t; e < all; e += T) {
      const uint32_t j = divide(e, n, a.n_inv), r = e - j * n;
      int32_t x, y;
      bool tail;
      entry(a, s, r, j, c0 + j, x, y, tail);
      if (x == y && !tail) continue;
      any = true;
      if (valid(x)) {
        add_here(delta + x, -1);
        max_here(mark + x, (int32_t)(n - r));
      }
      if (valid(y)) {
        if (tail) max_here(mark + y, (int32_t)(kWriter + n - r));
        else add_here(delta + y, 1);
      }
    }
    if (!__syncthreads_or(any)) continue;
    for (uint32_t e = t; e < all; e += T) {
      const uint32_t j = divide(e, n, a.n_inv), r = e - j * n;
      int32_t x, y;
      bool tail;
      entry(a, s, r, j, c0 + j, x, y, tail);
      if (x == y && !tail) continue;
      const Page at_x = page(x, valid(x)), at_y = page(y, tail && valid(y));
      freed += at_x.mark == (int32_t)(n - r) && at_x.holders == 0;
      if (tail) {   // the lowest of those that write keeps a page that nobody else holds
        const bool stays = !valid(y) || (at_y.mark == (int32_t)(kWriter + n - r) && at_y.holders == 0);
        const int32_t part = s.len[r] & ((1 << a.page_shift) - 1);
        if (!stays) atomicOr(&s.keep[r], kCopied);
        *reinterpret_cast<i32x4*>(a.copies + 4ull * r) = i32x4{y, y, stays ? 0 : part, 0};
      }
    }
  }
  if (blockIdx.x == 0)
    for (uint32_t r = t; r < n; r += T)
      if (!(s.keep[r] & kWrites)) *reinterpret_cast<i32x4*>(a.copies + 4ull * r) = i32x4{-1, -1, 0, 0};
  return block_sum<T>(freed, s.w);
}

// The second half.  ring: its head and count as they were; none: the first one has found a table that is
// none; before, freed: pages given back by the workgroups before and by all.
template <int T, int N>
__device__ __forceinline__ void fork_apply(const ForkArgs& a, ForkLds<T, N>& s, uint2 ring, bool none, uint32_t before,
                                           uint32_t freed) {
  constexpr uint32_t kPer = N / T;
  const uint32_t t = threadIdx.x, n = a.n_req, lane = t & 63, wave = t >> 6, cols = s.cols;
  const uint32_t first = blockIdx.x * T + t, step = a.grid * T;   // of the flat lists
  int32_t* const delta = a.refs + a.n_pages;
  int32_t* const mark = delta + a.n_pages;
  const uint32_t shift = a.page_shift, in_page = (1u << shift) - 1u;
  const uint32_t head = ring.x, count = ring.y;
  const uint32_t per_t = (n + T - 1) / T;
  uint32_t need[kPer], sum = 0;
#pragma unroll
  for (uint32_t i = 0; i < kPer; ++i) {
    const uint32_t r = t * per_t + i;
    need[i] = i < per_t && r < n ? s.need[r + 1] + ((s.keep[r] & kCopied) ? 1u : 0u) : 0u;
    sum = sat_add(sum, need[i]);
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t u = __shfl_up(sum, o);
    if (lane >= (uint32_t)o) sum = sat_add(sum, u);
  }
  if (lane == 63) s.w[wave] = sum;
  __syncthreads();
  uint32_t total = 0;
#pragma unroll
  for (uint32_t w = 0; w < T / 64; ++w) {
    if (w < wave) sum = sat_add(sum, s.w[w]);
    total = sat_add(total, s.w[w]);
  }
#pragma unroll
  for (int i = (int)kPer - 1; i >= 0; --i) {
    const uint32_t r = t * per_t + i;
    if (i < (int)per_t && r < n) {
      s.need[r + 1] = sum;
      sum -= need[i];
    }
  }
  const bool enough = !none && total <= count && (uint64_t)count + freed <= a.n_pages;
  __syncthreads();

  auto ring_at = [&](uint32_t j) {   // j <= n_pages
    const uint32_t i = head + j;
    return i >= a.n_pages ? i - a.n_pages : i;
  };
  auto valid = [&](int32_t p) { return (uint32_t)p < a.n_pages; };
  auto copied = [&](uint32_t r) { return (s.keep[r] & kCopied) != 0; };
  // the page that request r gets for its column c >= keep, or (c = keep - 1) for the copy
  auto fresh = [&](uint32_t r, uint32_t c, bool copy) {
    const uint32_t at = s.need[r] + (c + (copy ? 1u : 0u) - (s.keep[r] & kKeep));
    const int32_t p = at < s.need[r + 1] ? a.ring[ring_at(at)] : -1;
    return valid(p) ? p : -1;
  };

  // ---- the columns
  const Columns k = columns(a, s);
  uint32_t back = before;   // where this workgroup's pages go in the ring
  for (uint32_t c0 = k.begin; c0 < k.end && !none; c0 += k.width) {
    const uint32_t w = min(k.width, k.end - c0), all = w * n;
    fork_columns(a, s, c0, w);
    bool any = false;
    for (uint32_t e0 = 0; e0 < all; e0 += T) {
      const uint32_t e = e0 + t;
      int32_t x = -1, y = -1;
      bool tail = false;
      uint32_t r = 0;
      if (e < all) {
        const uint32_t j = divide(e, n, a.n_inv);
        r = e - j * n;
        entry(a, s, r, j, c0 + j, x, y, tail);
      }
      const bool moves = e < all && (x != y || tail);
      const Page now = moves && valid(x) ? page_now(a, x) : Page{0, 0};
      const bool gone = now.mark == (int32_t)(n - r) && now.holders == 0 && moves;
      any |= moves;
      if (__syncthreads_or(gone)) {
        uint32_t some;
        const uint32_t rank = block_rank<T>(gone, s.w, some);
        if (gone && enough) a.ring[ring_at(count + back + rank)] = x;
        back += some;
      }
    }
    any = __syncthreads_or(any);
    // the counts, and the call's own words back to zero
    if (any)
      for (uint32_t e = t; e < all; e += T) {
        const uint32_t j = divide(e, n, a.n_inv), r = e - j * n;
        int32_t x, y;
        bool tail;
        entry(a, s, r, j, c0 + j, x, y, tail);
        if (x == y && !tail) continue;
        const bool to = valid(y) && !(tail && copied(r));
        if (enough) {
          if (valid(x)) add_here(a.refs + x, -1);
          if (to) add_here(a.refs + y, 1);
        }
        if (valid(x)) delta[x] = mark[x] = 0;
        if (valid(y)) delta[y] = mark[y] = 0;
      }
    const uint32_t inv = 0xffffffffu / w;
    if (enough)
      for (uint32_t e = t; e < all; e += T) {
        const uint32_t r = divide(e, w, inv), j = e - r * w, c = c0 + j;
        int32_t x, y;
        bool tail;
        entry(a, s, r, j, c, x, y, tail);
        const uint32_t keep = s.keep[r] & kKeep, news = s.need[r + 1] - s.need[r];
        if (tail && copied(r)) {
          y = fresh(r, c, true);
          if (valid(y)) a.refs[y] = 1;
          a.copies[4ull * r + 1] = y;
        } else if (c >= keep) {
          const bool more = c - keep < news - (copied(r) ? 1u : 0u);
          if (!more) continue;   // (entries past the pages keep their values)
          y = fresh(r, c, copied(r));
          if (valid(y)) a.refs[y] = 1;
        }
        if (y != x) a.table[(uint64_t)r * a.max_pages + c] = y;
      }
  }
  if (enough)   // pages in columns that nobody held
    for (uint32_t e = first; e < total; e += step) {
      const uint32_t r = segment(s.need, n, e), own = copied(r) ? 1u : 0u, i = e - s.need[r];
      const uint32_t c = (s.keep[r] & kKeep) + i - own;
      if (i < own || c < cols) continue;
      const int32_t p = fresh(r, c, own != 0);
      if (valid(p)) a.refs[p] = 1;
      a.table[(uint64_t)r * a.max_pages + c] = p;
    }
  // ---- the rows, and the requests
  for (uint32_t i = first; i < a.m; i += step) {
    int32_t p = -1, q = -1;
    if (enough && i >= s.off[0] && i < s.off[n]) {
      const uint32_t r = segment(s.off, n, i);
      if (s.len[r] >= 0) {
        p = s.len[r] + (int32_t)(i - s.off[r]);
        const uint32_t c = (uint32_t)p >> shift;
        const bool copy = copied(r);
        const int32_t page = c < (s.keep[r] & kKeep) && !copy ? a.copies[4ull * r] : fresh(r, c, copy);
        if (valid(page)) q = (page << shift) | (p & (int32_t)in_page);
      }
    }
    a.pos[i] = p;
    a.slot[i] = q;
  }
  for (uint32_t r = first; r < n; r += step)
    a.kv_len[r] = enough && s.len[r] >= 0 ? s.len[r] + (int32_t)(s.off[r + 1] - s.off[r]) : -1;
  // what others read last: every workgroup is through with the old values
  if (none) {
    for (uint32_t r = first; r < n; r += step) *reinterpret_cast<i32x4*>(a.copies + 4ull * r) = i32x4{-1, -1, 0, 0};
    return;
  }
  __syncthreads();
  if (a.grid > 1) {
    if (t == 0) {
      uint32_t* const ticket = reinterpret_cast<uint32_t*>(a.state + 2);
      s.last = __hip_atomic_fetch_add(ticket, kTicket, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
               (a.grid - 1) * kTicket;
      if (s.last) __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (!s.last) return;
  }
  if (!enough) {   // nothing has changed
    for (uint32_t r = t; r < n; r += T) *reinterpret_cast<i32x4*>(a.copies + 4ull * r) = i32x4{-1, -1, 0, 0};
    return;
  }
  for (uint32_t r = t; r < n; r += T)
    if (s.len[r] >= 0) a.held[r] = (int32_t)((s.keep[r] & kKeep) + s.need[r + 1] - s.need[r] - (copied(r) ? 1u : 0u));
  if (t == 0) {
    a.state[0] = (int32_t)ring_at(total);
    a.state[1] = (int32_t)(count - total + freed);
  }
}

__device__ __forceinline__ bool no_ring(const ForkArgs& a) {
  const int32_t head = a.state[0], count = a.state[1];
  return head < 0 || (uint32_t)head >= a.n_pages || count < 0 || (uint32_t)count > a.n_pages || a.state[2] != 0;
}

template <int T, int N>
__global__ __launch_bounds__(T) void k_fork_look(ForkArgs a) {
  __shared__ ForkLds<T, N> s;
  uint32_t* const counts = reinterpret_cast<uint32_t*>(a.refs) + 5ull * a.n_pages;
  const bool state = no_ring(a), none = fork_requests(a, s) || state;
  if (blockIdx.x == 0 && threadIdx.x == 0) counts[kForkWG] = none;
  if (none) return;
  const uint32_t freed = fork_look(a, s);
  if (threadIdx.x == 0) counts[blockIdx.x] = freed;
}

template <int T, int N>
__global__ __launch_bounds__(T) void k_fork_apply(ForkArgs a) {
  static_assert(T >= (int)kForkWG, "a thread per workgroup's count");
  __shared__ ForkLds<T, N> s;
  const uint32_t* const counts = reinterpret_cast<const uint32_t*>(a.refs) + 5ull * a.n_pages;
  const uint32_t t = threadIdx.x, v = t < a.grid ? counts[t] : 0u, n = a.n_req;
  const bool none = counts[kForkWG] != 0;   // the first kernel has left everything as it was
  const uint2 ring = {(uint32_t)a.state[0], (uint32_t)a.state[1]};
  if (t < 2) s.sum[t] = 0;
  fork_requests(a, s);
  for (uint32_t r = t; r < n; r += T)
    if ((s.keep[r] & kWrites) && !none && a.copies[4ull * r + 2] > 0) s.keep[r] |= kCopied;
  uint32_t before = t < blockIdx.x ? v : 0u, freed = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    before += __shfl_xor(before, o);
    freed += __shfl_xor(freed, o);
  }
  if ((t & 63) == 0 && t < a.grid) {
    atomicAdd(&s.sum[0], before);
    atomicAdd(&s.sum[1], freed);
  }
  __syncthreads();
  fork_apply(a, s, ring, none, s.sum[0], s.sum[1]);
}

template <int T, int N>
__global__ __launch_bounds__(T) void k_fork_one(ForkArgs a) {
  __shared__ ForkLds<T, N> s;
  const uint2 ring = {(uint32_t)a.state[0], (uint32_t)a.state[1]};
  const bool state = no_ring(a), none = fork_requests(a, s) || state;
  const uint32_t freed = none ? 0u : fork_look(a, s);
  __syncthreads();
  fork_apply(a, s, ring, none, 0u, freed);
}

// ------------------------------------------------------------------------------- the copies
// A workgroup takes kCopyBytes of one page of K or V of one layer, 16 bytes a thread at a time
// and all reads before the first write, past the caches: what is copied here is read again after
// a layer's other work at the soonest.  Bound by HBM: 24 pages of 64 layers (201 MB read and written) in 38 us,
// 5.3 TB/s; with cached loads and stores 44 us, with 32 KB a workgroup 65 us.
constexpr uint32_t kCopyT = 256, kCopyBytes = 16384, kCopyV = kCopyBytes / 16 / kCopyT;

__global__ __launch_bounds__(kCopyT) void k_kv_copy(CopyArgs a) {
  const int32_t* const c = a.copies + 4ull * blockIdx.x;
  const int32_t src = c[0], dst = c[1], tokens = c[2];
  if (tokens <= 0 || src == dst || (uint32_t)src >= a.n_pages || (uint32_t)dst >= a.n_pages) return;
  const bool of_v = blockIdx.z & 1;
  const uint32_t part = blockIdx.z >> 1, page = 1u << a.page_shift;
  const uint32_t here = min(((uint32_t)tokens + 15u) & ~15u, page);
  uint8_t* const base = (uint8_t*)(of_v ? a.v[blockIdx.y] : a.k[blockIdx.y]);
  const u32x4* const from = reinterpret_cast<const u32x4*>(base + (uint64_t)src * a.page_bytes);
  u32x4* const to = reinterpret_cast<u32x4*>(base + (uint64_t)dst * a.page_bytes);
  auto e_of = [&](uint32_t i) { return part * (kCopyBytes / 16) + i * kCopyT + threadIdx.x; };
  u32x4 x[kCopyV];
  bool on[kCopyV];
#pragma unroll
  for (uint32_t i = 0; i < kCopyV; ++i) {
    const uint32_t e = e_of(i), place = of_v ? e << a.vec_shift : e >> a.key_shift;
    on[i] = e < a.page_bytes / 16 && (place & (page - 1u)) < here;
    if (on[i]) x[i] = __builtin_nontemporal_load(from + e);
  }
#pragma unroll
  for (uint32_t i = 0; i < kCopyV; ++i)
    if (on[i]) __builtin_nontemporal_store(x[i], to + e_of(i));
}

// ---------------------------------------------------------------------- clearing a range
// Three launches: the workgroups' counts; ranks of the pages that move and of the free pages
// outside, the new ring; then the moves, the counts and the tables' names.  One launch of one
// workgroup for small pools: a third of the time at 401 pages (us: 6.1 for 16), the same at 1500 pages,
// twice the time at 8000.  Bound by latency.
constexpr uint32_t kClearOnePages = 2048, kClearOnePlaces = 8192;
struct Clear {   // free pages outside the range and pages in use in it: all, and those before the workgroup's
  uint32_t out, in, out_before, in_before;
};

template <int T>
__device__ __forceinline__ Clear clear_counts(const ClearArgs& a, uint32_t* s_w) {   // s_w [4 * T / 64]
  const uint32_t* const counts = reinterpret_cast<const uint32_t*>(a.refs) + 5ull * a.n_pages;
  const uint32_t t = threadIdx.x;
  uint32_t v[4] = {0, 0, 0, 0};
  if (t < a.blocks) {
    v[0] = counts[2 * t];
    v[1] = counts[2 * t + 1];
    if (t < blockIdx.x) {
      v[2] = v[0];
      v[3] = v[1];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v[i] += __shfl_xor(v[i], o);
    if ((t & 63) == 0) s_w[4 * (t >> 6) + i] = v[i];
  }
  __syncthreads();
  Clear n{0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < T / 64; ++w) {
    n.out += s_w[4 * w];
    n.in += s_w[4 * w + 1];
    n.out_before += s_w[4 * w + 2];
    n.in_before += s_w[4 * w + 3];
  }
  __syncthreads();
  return n;
}

// Pages x0 .. x1 - 1: free ones outside (x), in use inside (y).
template <int T>
__device__ __forceinline__ uint2 clear_count(const ClearArgs& a, uint32_t x0, uint32_t x1, uint32_t* s_w) {
  uint32_t out = 0, in = 0;
  for (uint32_t x = x0 + threadIdx.x; x < x1; x += T) {
    const bool inside = x - a.first < a.n_clear, live = a.refs[x] > 0;
    out += !inside && !live;
    in += inside && live;
  }
  out = block_sum<T>(out, s_w);
  in = block_sum<T>(in, s_w);
  return uint2{out, in};
}

template <int T>
__device__ __forceinline__ void clear_rank(const ClearArgs& a, const Clear& n, uint32_t x0, uint32_t x1, uint32_t* s_w) {
  if (n.in > n.out) return;
  int32_t* const rank = a.refs + 3ull * a.n_pages;
  int32_t* const target = rank + a.n_pages;
  uint32_t out = n.out_before, in = n.in_before;
  for (uint32_t x = x0; x < x1; x += T) {
    const uint32_t p = x + threadIdx.x;
    const bool inside = p - a.first < a.n_clear, live = p < x1 && a.refs[p] > 0;
    uint32_t some, k = block_rank<T>(p < x1 && !inside && !live, s_w, some);
    if (p < x1 && !inside && !live) {
      if (out + k < n.in) target[out + k] = (int32_t)p;
      else a.ring[out + k - n.in] = (int32_t)p;
    }
    out += some;
    k = block_rank<T>(inside && live, s_w, some);
    if (p < x1 && inside) {
      rank[p] = live ? (int32_t)(in + k) : -1;
      a.ring[n.out - n.in + (p - a.first)] = (int32_t)p;
    }
    in += some;
  }
}

template <int T>
__device__ __forceinline__ void clear_move(const ClearArgs& a, const Clear& n) {
  const bool enough = n.in <= n.out;
  const int32_t* const rank = a.refs + 3ull * a.n_pages;
  const int32_t* const target = rank + a.n_pages;
  const uint32_t t = threadIdx.x;
  auto moved = [&](uint32_t p) {   // where page p of the range went
    const int32_t k = rank[p];
    return (uint32_t)k < n.in ? target[k] : -1;
  };
  const uint64_t wg = (uint64_t)blockIdx.y * gridDim.x + blockIdx.x, all = (uint64_t)gridDim.x * gridDim.y;
  for (uint64_t i = wg * T + t; i < a.n_clear; i += all * T) {
    const uint32_t p = a.first + (uint32_t)i;
    const int32_t to = enough ? moved(p) : -1;
    if (to >= 0) {
      a.refs[to] = a.refs[p];
      a.refs[p] = 0;
    }
    *reinterpret_cast<i32x4*>(a.moves + 4 * i) =
        to >= 0 ? i32x4{(int32_t)p, to, (int32_t)a.page_size, 0} : i32x4{-1, -1, 0, 0};
  }
  if (enough) {   // a wave takes 64 places of a row
    const uint32_t wave = blockIdx.y * (T / 64) + (t >> 6), lane = t & 63, waves = gridDim.y * (T / 64);
    for (uint32_t r = blockIdx.x; r < a.max_req; r += gridDim.x) {
      const int32_t held = a.held[r];
      if (held < 0 || (uint32_t)held > a.max_pages) continue;
      int32_t* const row = a.table + (uint64_t)r * a.max_pages;
      for (uint32_t c = wave * 64 + lane; c < (uint32_t)held; c += waves * 64) {
        const int32_t p = row[c];
        if ((uint32_t)p >= a.n_pages || (uint32_t)p - a.first >= a.n_clear) continue;
        const int32_t to = moved((uint32_t)p);
        if (to >= 0) row[c] = to;
      }
    }
  }
  if (wg == 0 && t == 0) {
    *a.moved = enough ? (int32_t)n.in : -1;
    if (enough) {
      a.state[0] = 0;
      a.state[1] = (int32_t)(n.out - n.in + a.n_clear);
    }
  }
}

__global__ __launch_bounds__(256) void k_clear_count(ClearArgs a) {
  __shared__ uint32_t s_w[4];
  uint32_t* const counts = reinterpret_cast<uint32_t*>(a.refs) + 5ull * a.n_pages;
  const uint32_t x0 = blockIdx.x * a.per;
  const uint2 n = clear_count<256>(a, x0, min(a.n_pages, x0 + a.per), s_w);
  if (threadIdx.x == 0) {
    counts[2 * blockIdx.x] = n.x;
    counts[2 * blockIdx.x + 1] = n.y;
  }
}

__global__ __launch_bounds__(256) void k_clear_rank(ClearArgs a) {
  __shared__ uint32_t s_w[16];
  const Clear n = clear_counts<256>(a, s_w);
  const uint32_t x0 = blockIdx.x * a.per;
  clear_rank<256>(a, n, x0, min(a.n_pages, x0 + a.per), s_w);
}

__global__ __launch_bounds__(256) void k_clear_move(ClearArgs a) {
  __shared__ uint32_t s_w[16];
  clear_move<256>(a, clear_counts<256>(a, s_w));
}

__global__ __launch_bounds__(1024) void k_clear_one(ClearArgs a) {
  __shared__ uint32_t s_w[16];
  const uint2 c = clear_count<1024>(a, 0, a.n_pages, s_w);
  const Clear n{c.x, c.y, 0, 0};
  clear_rank<1024>(a, n, 0, a.n_pages, s_w);
  __syncthreads();
  clear_move<1024>(a, n);
}

}  // namespace

hipError_t launch_kv_fork(const ForkArgs& given, hipStream_t s) {
  ForkArgs a = given;
  // One workgroup for up to 1024 places of the tables, or rows, else one for every 512, so that a thread takes
  // one place, two behind 256 workgroups (us for 96 beams of 515 places: 20.7 with 1024 places and 256
  // threads, 17.0 with 512 and 256, 16.0 with 512 threads; 8 requests of 96 in one launch 11.6, in two 13.4; 4
  // requests of 24 with 256 threads 8.5, with 512 9.1)
  const uint64_t places = (uint64_t)a.n_req * a.max_pages, work = places > a.m ? places : a.m;
  const uint64_t wg = work <= 1024 && a.n_req <= 512 ? 1 : (work + 511) / 512;
  a.grid = (uint32_t)(wg > kForkWG ? kForkWG : wg);
  a.n_inv = 0xffffffffu / a.n_req;
  a.at_once = kEntries / a.n_req;
  const dim3 grid(a.grid);
  if (a.grid == 1 && work <= 256) {
    hipLaunchKernelGGL((k_fork_one<256, 256>), grid, dim3(256), 0, s, a);
  } else if (a.grid == 1 && a.n_req <= 512) {
    hipLaunchKernelGGL((k_fork_one<512, 512>), grid, dim3(512), 0, s, a);
  } else if (a.n_req <= 512) {
    hipLaunchKernelGGL((k_fork_look<512, 512>), grid, dim3(512), 0, s, a);
    hipLaunchKernelGGL((k_fork_apply<512, 512>), grid, dim3(512), 0, s, a);
  } else {
    hipLaunchKernelGGL((k_fork_look<1024, 4096>), grid, dim3(1024), 0, s, a);
    hipLaunchKernelGGL((k_fork_apply<1024, 4096>), grid, dim3(1024), 0, s, a);
  }
  return hipGetLastError();
}

hipError_t launch_kv_copy(const CopyArgs& a, uint32_t n_copies, uint32_t n_layers, hipStream_t s) {
  const uint32_t parts = (a.page_bytes + kCopyBytes - 1) / kCopyBytes;
  hipLaunchKernelGGL(k_kv_copy, dim3(n_copies, n_layers, 2 * parts), dim3(kCopyT), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_kv_compact(const ClearArgs& given, hipStream_t s) {
  ClearArgs a = given;
  if (a.n_pages <= kClearOnePages && (uint64_t)a.max_req * a.max_pages <= kClearOnePlaces) {
    hipLaunchKernelGGL(k_clear_one, dim3(1), dim3(1024), 0, s, a);
    return hipGetLastError();
  }
  a.per = (a.n_pages + 255) / 256;
  a.per = a.per < 256 ? 256 : a.per;
  a.blocks = (a.n_pages + a.per - 1) / a.per;
  hipLaunchKernelGGL(k_clear_count, dim3(a.blocks), dim3(256), 0, s, a);
  hipLaunchKernelGGL(k_clear_rank, dim3(a.blocks), dim3(256), 0, s, a);
  const uint32_t x = a.max_req < 256 ? a.max_req : 256, most = (a.max_pages + 255) / 256, y = 1024 / x;
  hipLaunchKernelGGL(k_clear_move, dim3(x, y < most ? y : most), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace w12
