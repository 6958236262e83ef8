// The 4-bit KV cache outside attention: page tables and slot maps from request
// lengths, the quantising write of new rows, and the read-back.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kv_internal.h"

namespace moe {

namespace {

constexpr int kTableThreads = 512;

// Exclusive block-wide sums of two values per thread (kTableThreads threads);
// totals in *ta, *tb.  Sums saturate nowhere: 64 bits.
__device__ __forceinline__ void block_exclusive2(long long& a, long long& b, long long* ta, long long* tb,
                                                 long long* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kWarps = kTableThreads / 32;
  long long ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long xa = __shfl_up_sync(0xffffffffu, ia, o), xb = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) {
      ia += xa;
      ib += xb;
    }
  }
  __syncthreads();  // scratch may still be read by the previous call
  if (lane == 31) {
    scratch[warp] = ia;
    scratch[kWarps + warp] = ib;
  }
  __syncthreads();
  long long pa = 0, pb = 0, sa = 0, sb = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const long long xa = scratch[w], xb = scratch[kWarps + w];
    if (w < warp) {
      pa += xa;
      pb += xb;
    }
    sa += xa;
    sb += xb;
  }
  a = pa + ia - a;
  b = pb + ib - b;
  *ta = sa;
  *tb = sb;
}

// Page tables and slot maps (kv_mxfp4_page_tables).  Latency-bound: a few KB
// of lengths in, 8 bytes per new token out (8 requests 3.9 us, 1,000 with 36,000
// new tokens 7.1).  Every CTA redoes the two prefix
// sums over the requests (tokens, then pages) in shared memory, so one launch
// needs no grid-wide step; the CTAs then share the tokens and the finished
// requests.  A token whose position starts a page that its request does not
// hold yet takes the page off the ring and writes the table entry.
__global__ void __launch_bounds__(kTableThreads) page_tables_kernel(const PageTableArgs a) {
  extern __shared__ int32_t sm[];
  int32_t* start = sm;              // [R + 1] first token of each request
  int32_t* cached = start + a.R + 1;  // [R]
  int32_t* ofs = cached + a.R;      // [R] ring offset of its first new page; -1: refused
  __shared__ long long scratch[2 * (kTableThreads / 32)];
  __shared__ int taken_sum;
  const int tid = threadIdx.x, R = a.R;
  if (tid == 0) taken_sum = 0;
  const int page = 1 << a.page_shift;
  constexpr long long kMost = 0x7FFFFFFF;  // tokens of a request
  const int per = (R + kTableThreads - 1) / kTableThreads;  // consecutive requests of this thread
  const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
  const int head = ((a.state[0] % a.ring_size) + a.ring_size) % a.ring_size;
  const int avail = min(max(a.state[1], 0), a.ring_size);

  for (int r = tid; r < R; r += kTableThreads) {
    cached[r] = max(a.cached[r], 0);
    ofs[r] = a.added[r];
  }
  __syncthreads();
  long long tok = 0, zero = 0, total, unused;
  for (int r = r0; r < r1; ++r) tok += max(ofs[r], 0);
  block_exclusive2(tok, zero, &total, &unused, scratch);
  // pages needed by requests that fit otherwise, pages given back
  long long need = 0, gone = 0;
  {
    long long t = tok;
    for (int r = r0; r < r1; ++r) {
      const int n = ofs[r];
      const long long have = ((long long)cached[r] + page - 1) >> a.page_shift;
      const long long all = ((long long)cached[r] + max(n, 0) + page - 1) >> a.page_shift;
      if (n < 0) gone += min(have, (long long)a.max_blocks);
      else if (t + n <= a.max_tokens && all <= a.max_blocks && (long long)cached[r] + n <= kMost) need += all - have;
      t += max(n, 0);
    }
  }
  long long need_all, gone_all;
  block_exclusive2(need, gone, &need_all, &gone_all, scratch);
  const bool first = blockIdx.x == 0;
  long long taken = 0;  // pages taken by this thread's requests
  for (int r = r0; r < r1; ++r) {
    const int n = ofs[r];
    const long long have = ((long long)cached[r] + page - 1) >> a.page_shift;
    const long long all = ((long long)cached[r] + max(n, 0) + page - 1) >> a.page_shift;
    start[r] = (int)min(tok, 0x7FFFFFFFll);
    int seq = 0, o = -1;
    if (n < 0) {
      // finished: its pages go to the ring's end, this thread's share of the
      // CTAs' work below; the offset is kept as -2 - offset
      // (within the ring's size where the requests claim more pages than it can hold)
      o = -2 - (int)(gone >> 30 ? gone % a.ring_size : gone);
      gone += min(have, (long long)a.max_blocks);
    } else {
      bool ok = tok + n <= a.max_tokens && all <= a.max_blocks && (long long)cached[r] + n <= kMost;
      const long long want = ok ? all - have : 0;
      ok = ok && (want == 0 || need + want <= avail);
      if (ok) {
        o = (int)need;
        taken += want;
      }
      need += want;
      seq = ok ? cached[r] + n : -1;
      tok += n;
    }
    ofs[r] = o;
    if (first) {
      a.seq_lens[r] = seq;
      a.query_start[r] = start[r];
    }
  }
  if (tid == 0) start[R] = (int)min(total, 0x7FFFFFFFll);
  const int taken_warp = __reduce_add_sync(0xffffffffu, (int)taken);  // at most the free pages in all
  if ((tid & 31) == 0 && taken_warp > 0) atomicAdd(&taken_sum, taken_warp);
  __syncthreads();  // the shared arrays are complete
  const int taken_all = taken_sum;
  if (first && tid == 0) {
    a.query_start[R] = start[R];
    const uint32_t at = (uint32_t)head + (uint32_t)taken_all;
    a.state_out[0] = (int)(at >= (uint32_t)a.ring_size ? at - (uint32_t)a.ring_size : at);
    a.state_out[1] = (int)(avail - taken_all + gone_all);
  }

  const uint32_t nt = gridDim.x * kTableThreads;
  // (unsigned: the step past the last of up to 2^31 - 1 tokens leaves an int)
  for (uint32_t ut = blockIdx.x * kTableThreads + tid; ut < (uint32_t)a.max_tokens; ut += nt) {
    const int t = (int)ut;
    int slot = -1, pos = -1;
    if (t < start[R]) {
      int lo = 0, hi = R;  // start[lo] <= t < start[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= t) lo = mid;
        else hi = mid;
      }
      pos = (int)min((uint32_t)cached[lo] + (uint32_t)(t - start[lo]), (uint32_t)kMost);  // (more: refused)
      const int o = ofs[lo];
      if (o >= 0) {
        const int b = pos >> a.page_shift;
        const int have = (int)(((long long)cached[lo] + page - 1) >> a.page_shift);
        int32_t* entry = a.table + (size_t)lo * a.max_blocks + b;
        int pg;
        if (b < have) {
          pg = *entry;
        } else {
          // (head < ring size, o + (b - have) < free pages <= ring size)
          const uint32_t at = (uint32_t)head + (uint32_t)(o + (b - have));
          pg = a.ring[at >= (uint32_t)a.ring_size ? at - (uint32_t)a.ring_size : at];
          if ((pos & (page - 1)) == 0) *entry = pg;
        }
        slot = (int)(((long long)pg << a.page_shift) + (pos & (page - 1)));
      }
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
  }
  // finished requests: one warp each
  const int lane = tid & 31, nw = gridDim.x * (kTableThreads / 32);
  for (int r = blockIdx.x * (kTableThreads / 32) + (tid >> 5); r < R; r += nw) {
    const int o = ofs[r];
    if (o > -2) continue;
    const int have = (int)min(((long long)cached[r] + page - 1) >> a.page_shift, (long long)a.max_blocks);
    const int32_t* row = a.table + (size_t)r * a.max_blocks;
    const int to = (int)(((long long)head + avail + (-2 - o)) % a.ring_size);
    // eight pages a lane at a time (one by one, each waits for the last: 11.5 us
    // for 1,000 requests of which 50 finish)
    for (int b0 = 0; b0 < have; b0 += 256) {
      int32_t pg[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int b = b0 + 32 * i + lane;
        pg[i] = b < have ? row[b] : 0;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int b = b0 + 32 * i + lane;
        if (b < have) {
          const uint32_t at = (uint32_t)to + (uint32_t)b % (uint32_t)a.ring_size;
          a.ring[at >= (uint32_t)a.ring_size ? at - (uint32_t)a.ring_size : at] = pg[i];
        }
      }
    }
  }
}

// Byte of a record that holds K row byte j (a multiple of 4) of token t, and V row byte j (a multiple of 2).
template <int D>
__device__ __forceinline__ int k_byte(int t, int j) {
  constexpr int NB = D / 32;
  return ((t * 4 + ((j >> 2) & 3)) * NB + (j >> 4)) * 4;
}
template <int D>
__device__ __forceinline__ int v_byte(int t, int j) {
  constexpr int NB = D / 32;
  return 8 * D + ((((((t >> 3) * 8 + ((j >> 1) & 7)) * 4 + ((t >> 1) & 3)) * 2 + (t & 1)) * NB) + (j >> 4)) * 2;
}

// MXFP4 codes and scale byte of a lane's 8 values of a 32-value block (4
// lanes; the whole warp calls it), any float inputs: a NaN makes the block's
// byte 255 (its finite values keep their codes, the rest get 0), an infinity
// saturates on the largest finite scale (byte 252).
__device__ __forceinline__ void kv_quant8(float (&v)[8], uint32_t& codes, uint32_t& sbyte) {
  float m = 0.f;
  bool odd = false;  // infinite or NaN
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    m = fmaxf(m, fabsf(v[q]));
    odd |= !(fabsf(v[q]) <= 3.402823466e38f);
  }
  bool nan = false;
  if (__any_sync(0xffffffffu, odd)) {  // rare
#pragma unroll
    for (int q = 0; q < 8; ++q) nan |= v[q] != v[q];
    nan |= (bool)__shfl_xor_sync(0xffffffffu, (int)nan, 1);
    nan |= (bool)__shfl_xor_sync(0xffffffffu, (int)nan, 2);
    if (nan) {
      m = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (!(fabsf(v[q]) <= 3.402823466e38f)) v[q] = 0.f;
        m = fmaxf(m, fabsf(v[q]));
      }
    }
  }
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const uint32_t s = min(mx_scale_byte(m), 252u);
  const float rcp = __uint_as_float((254u - s) << 23);  // 2^(127 - s)
  float r[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) r[q] = v[q] * rcp;
  codes = f32x8_to_e2m1x8(r);
  sbyte = nan ? 255u : s;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The same of eight bf16 values as they are, two at a time: magnitudes compare
// as integers (NaN above infinity above all), the scaling is exact in bf16
// (unless far below 0.25, which rounds to 0 either way).
__device__ __forceinline__ void kv_quant8(const uint4& u, uint32_t& codes, uint32_t& sbyte) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  const uint32_t mm = max_u16x2(max_u16x2(u.x & kAbs, u.y & kAbs), max_u16x2(u.z & kAbs, u.w & kAbs));
  uint32_t m = max(mm & 0xFFFFu, mm >> 16);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  if (__any_sync(0xffffffffu, m >= 0x7F80u)) {  // infinite or NaN, rare
    float x[8] = {bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y),
                  bf16_lo(u.z), bf16_hi(u.z), bf16_lo(u.w), bf16_hi(u.w)};
    kv_quant8(x, codes, sbyte);
    return;
  }
  const uint32_t eb = m >> 7;
  sbyte = eb > 2u ? eb - 2u : 0u;
  const uint32_t rcp = (254u - sbyte) * 0x00800080u;  // 2^(127 - s), twice
  const uint32_t a = mul_bf16x2(u.x, rcp), b = mul_bf16x2(u.y, rcp), c = mul_bf16x2(u.z, rcp), d = mul_bf16x2(u.w, rcp);
  const float r[8] = {bf16_lo(a), bf16_hi(a), bf16_lo(b), bf16_hi(b), bf16_lo(c), bf16_hi(c), bf16_lo(d), bf16_hi(d)};
  codes = f32x8_to_e2m1x8(r);
}

template <bool F32>
struct Raw8;  // eight input values as loaded
template <>
struct Raw8<false> {
  uint4 u;
  __device__ __forceinline__ void load(const void* p, long long at) {
    u = __ldcs(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + at));
  }
  __device__ __forceinline__ void quant(bool live, uint32_t& codes, uint32_t& sbyte) const {
    kv_quant8(live ? u : make_uint4(0u, 0u, 0u, 0u), codes, sbyte);
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(w[i]);
      x[2 * i + 1] = bf16_hi(w[i]);
    }
  }
  // the values of lane ``src``
  __device__ __forceinline__ Raw8 of_lane(int src) const {
    return Raw8{make_uint4(__shfl_sync(0xffffffffu, u.x, src), __shfl_sync(0xffffffffu, u.y, src),
                           __shfl_sync(0xffffffffu, u.z, src), __shfl_sync(0xffffffffu, u.w, src))};
  }
};
template <>
struct Raw8<true> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, long long at) {
    const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + at);
    a = __ldcs(q);
    b = __ldcs(q + 1);
  }
  __device__ __forceinline__ void quant(bool live, uint32_t& codes, uint32_t& sbyte) const {
    float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = live ? x[q] : 0.f;
    kv_quant8(x, codes, sbyte);
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ Raw8 of_lane(int src) const {
    Raw8 r;
    r.a = make_float4(__shfl_sync(0xffffffffu, a.x, src), __shfl_sync(0xffffffffu, a.y, src),
                      __shfl_sync(0xffffffffu, a.z, src), __shfl_sync(0xffffffffu, a.w, src));
    r.b = make_float4(__shfl_sync(0xffffffffu, b.x, src), __shfl_sync(0xffffffffu, b.y, src),
                      __shfl_sync(0xffffffffu, b.z, src), __shfl_sync(0xffffffffu, b.w, src));
    return r;
  }
};

// Rows a thread keeps in flight, and CTAs per SM that the rows are dealt to:
// enough bytes under way to cover the chain slot -> row -> store (append and
// gather of 16,384 x 8 x 128: 2 rows, 6 / 8 / 16 CTAs 33.1 / 31.9 / 33.3 us; 4 rows,
// 3 / 4 / 8 CTAs 34.6 / 33.3 / 34.2; 8 rows, 2 CTAs 37.4).
constexpr int kRowsInFlight = 2, kRowCtas = 8;

// A walk over rows (token, head) in steps of ``step`` rows: one division each of
// the first row and of the step, none a row (64-bit divisions took a third of
// the instructions of both kernels).
struct RowWalk {
  int tok, head, dtok, dhead, heads;
  __device__ __forceinline__ RowWalk(long long row, long long step, int heads_) : heads(heads_) {
    tok = (int)(row / heads);
    head = (int)(row - (long long)tok * heads);
    dtok = (int)(step / heads);
    dhead = (int)(step - (long long)dtok * heads);
  }
  __device__ __forceinline__ void next() {
    tok += dtok;
    head += dhead;
    if (head >= heads) {
      head -= heads;
      ++tok;
    }
  }
};

// Writes a lane's codes of a K and a V row and the row's scale bytes to its slot
// (the whole warp calls it; ``live``: the slot exists).  Neighbouring blocks' lanes
// trade halves of their V words, so that each writes four bytes of one lane's operand.
template <int D>
__device__ __forceinline__ void store_row(const KvView& c, int slot, int head, bool live, const uint32_t (&code)[2],
                                          const uint32_t (&sb)[2]) {
  constexpr int L = D / 8, NB = D / 32;
  const int sub = threadIdx.x % L, b = sub >> 2, t4 = sub & 3;
  // V: lanes of blocks b and b ^ 1 hold bytes 2 t4 (lower half) and 2 t4 + 1
  // (upper) of their blocks; even b takes the lower halves of both, odd b the upper
  const uint32_t theirs = __shfl_xor_sync(0xffffffffu, code[1], 4);
  const uint32_t vw = (b & 1) ? prmt(theirs, code[1], 0x7632u) : prmt(code[1], theirs, 0x5410u);
  if (live) {
    const int off = slot & ((1 << c.page_shift) - 1), t = off & 15;
    uint8_t* rec = c.data + c.record(slot >> c.page_shift, head, off >> 4);
    *reinterpret_cast<uint32_t*>(rec + k_byte<D>(t, 4 * sub)) = code[0];
    *reinterpret_cast<uint32_t*>(rec + v_byte<D>(t, 4 * t4 + 2 * (b & 1) + 16 * (b & ~1))) = vw;
    if (t4 < 2) rec[16 * D + t4 * (D / 2) + t * NB + b] = (uint8_t)sb[t4];
  }
}

// Quantising write (kv_mxfp4_append).  HBM-bound: 2 or 4 bytes read and 17/32
// byte written per value (16,384 x 8 x 128, written and read back: 31.4 us, 5.4
// TB/s of the bytes that both must move).  D / 8 lanes take a token's K and V row of one head;
// the loop bounds are uniform per warp, so every lane reaches the shuffles.
template <int D, bool F32>
__global__ void __launch_bounds__(256) kv_append_kernel(const KvView c, const void* __restrict__ k,
                                                        const void* __restrict__ v, long long ks, long long vs, int N,
                                                        const int32_t* __restrict__ slots) {
  constexpr int L = D / 8;  // lanes per row
  const long long rows = (long long)N * c.heads;
  const int sub = threadIdx.x % L;
  const long long step = (long long)gridDim.x * (256 / L), first = (long long)blockIdx.x * (256 / L);
  RowWalk at(first + threadIdx.x / L, step, c.heads);
  for (long long w0 = first; w0 < rows; w0 += step * kRowsInFlight) {
    Raw8<F32> raw[kRowsInFlight][2];
    int slot[kRowsInFlight], head[kRowsInFlight];
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
      const int tok = at.tok;
      head[i] = at.head;
      slot[i] = -1;
      if (w0 + i * step + threadIdx.x / L < rows) {
        slot[i] = slots[tok];
        const int in = head[i] * D + 8 * sub;
        raw[i][0].load(k, (long long)tok * ks + in);
        raw[i][1].load(v, (long long)tok * vs + in);
      }
      at.next();
    }
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
      if (w0 + i * step >= rows) break;  // (uniform per CTA)
      const bool live = slot[i] >= 0 && (slot[i] >> c.page_shift) < c.num_pages;
      uint32_t code[2], sb[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) raw[i][w].quant(live, code[w], sb[w]);
      store_row<D>(c, slot[i], head[i], live, code, sb);
    }
  }
}

// The rotation of a lane's 8 values of a row, x, by the position's cosines and
// sines: pairs (i, i + rot / 2) of the row, or with PAIRS (2i, 2i + 1).  Float32,
// every product and sum rounded (so that codes of the rotated keys do not depend on how a
// compiler contracts them).  Elements from ``rot`` on stay.
struct Turn {
  float c[8], s[8];  // of the lane's elements, the sine with the sign that the partner's product takes
  int partner;       // lane that holds the partners
  bool on;
};
template <int D, bool PAIRS>
__device__ __forceinline__ Turn load_turn(const float* __restrict__ row, int rot) {
  constexpr int L = D / 8;
  const int sub = threadIdx.x % L, half = rot >> 1;
  Turn r;
  r.on = 8 * sub < rot;
  r.partner = threadIdx.x & 31;
  if (PAIRS) {
    float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r.on && row) {
      c = __ldg(reinterpret_cast<const float4*>(row + 4 * sub));
      s = __ldg(reinterpret_cast<const float4*>(row + half + 4 * sub));
    }
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      r.c[2 * k] = r.c[2 * k + 1] = cc[k];
      r.s[2 * k] = -ss[k];
      r.s[2 * k + 1] = ss[k];
    }
  } else {
    const bool upper = 8 * sub >= half;
    if (r.on) r.partner += upper ? -(half >> 3) : half >> 3;
    const int i = upper ? 8 * sub - half : 8 * sub;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r.on && row) {
        c = __ldg(reinterpret_cast<const float4*>(row + i) + k);
        s = __ldg(reinterpret_cast<const float4*>(row + half + i) + k);
      }
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r.c[4 * k + j] = cc[j];
        r.s[4 * k + j] = upper ? ss[j] : -ss[j];
      }
    }
  }
  return r;
}
// (the whole warp calls it)
template <bool PAIRS, bool F32>
__device__ __forceinline__ void turn8(const Turn& r, const Raw8<F32>& raw, float (&x)[8]) {
  float a[8], p[8];
  raw.values(a);
  if (PAIRS) {
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = a[k ^ 1];
  } else {
    raw.of_lane(r.partner).values(p);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = r.on ? __fadd_rn(__fmul_rn(a[k], r.c[k]), __fmul_rn(p[k], r.s[k])) : a[k];
}

// Rotated queries and the quantising write of rotated keys and of values
// (kv_mxfp4_append_rope).  HBM-bound: 2 or 4 bytes read a value, 2 bytes written of
// a query and 17/32 of a key or value (16,384 tokens of 28 / 4 heads of 128: bf16 50.1 us, 5.7
// TB/s, float32 72.3, 6.0; 32 tokens 2.8 us, one launch).  D / 8 lanes take a unit: up to kQueryRows
// query heads of one token, which share its cosines and sines, or the K and V row of
// one head.  Warps up to ``q_warps`` of the grid take queries, the others keys and
// values (the loop bounds are uniform per warp).
constexpr int kQueryRows = 4;
constexpr int rope_ctas(bool f32) { return f32 ? 2 : 3; }  // an SM: what its registers hold
template <int D, bool F32, bool PAIRS>
__global__ void __launch_bounds__(256, rope_ctas(F32)) kv_append_rope_kernel(const KvView c, const RopeArgs a, int q_warps) {
  constexpr int L = D / 8, W = 32 / L;  // lanes a unit, units a warp
  const int lane = threadIdx.x & 31, sub = lane % L;
  const int warp = blockIdx.x * 8 + (threadIdx.x >> 5), warps = gridDim.x * 8;
  const bool queries = warp < q_warps;
  const int per = queries ? (a.Hq + kQueryRows - 1) / kQueryRows : c.heads;  // units a token
  const long long units = (long long)a.N * per;
  const long long step = (long long)(queries ? q_warps : warps - q_warps) * W;
  long long w0 = (long long)(queries ? warp : warp - q_warps) * W;
  if (w0 >= units) return;
  RowWalk at(w0 + lane / L, step, per);
  for (; w0 < units; w0 += step, at.next()) {
    const bool there = w0 + lane / L < units;
    const int tok = at.tok;
    const int p0 = there ? a.positions[tok] : -1;
    const long long pos = (long long)p0 + a.position_offset;
    const bool known = p0 >= 0 && pos < a.max_positions;
    if (queries) {
      const int h0 = at.head * kQueryRows;
      Raw8<F32> raw[kQueryRows];
#pragma unroll
      for (int i = 0; i < kQueryRows; ++i)
        if (there && h0 + i < a.Hq) raw[i].load(a.q, (long long)tok * a.q_stride + (h0 + i) * D + 8 * sub);
      const Turn turn = load_turn<D, PAIRS>(known ? a.cos_sin + pos * a.rotary_dim : nullptr, a.rotary_dim);
#pragma unroll
      for (int i = 0; i < kQueryRows; ++i) {
        float x[8];
        turn8<PAIRS>(turn, raw[i], x);
        if (there && h0 + i < a.Hq) {
          uint4 o = make_uint4(f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]), f32x2_to_bf16x2(x[4], x[5]),
                               f32x2_to_bf16x2(x[6], x[7]));
          // padding: zeros; a position past the table: NaN
          if (!known) o.x = o.y = o.z = o.w = p0 < 0 ? 0u : 0x7FFF7FFFu;
          __stcs(reinterpret_cast<uint4*>(a.q_out + ((size_t)tok * a.Hq + h0 + i) * D + 8 * sub), o);
        }
      }
    } else {
      const int head = at.head, slot = there ? a.slots[tok] : -1;
      const bool live = slot >= 0 && (slot >> c.page_shift) < c.num_pages && p0 >= 0;
      Raw8<F32> raw[2];
      if (live) {
        raw[0].load(a.k, (long long)tok * a.k_stride + head * D + 8 * sub);
        raw[1].load(a.v, (long long)tok * a.v_stride + head * D + 8 * sub);
      }
      const Turn turn = load_turn<D, PAIRS>(known ? a.cos_sin + pos * a.rotary_dim : nullptr, a.rotary_dim);
      float x[8];
      turn8<PAIRS>(turn, raw[0], x);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = !live ? 0.f : known ? x[k] : __uint_as_float(0x7FC00000u);
      uint32_t code[2], sb[2];
      kv_quant8(x, code[0], sb[0]);
      raw[1].quant(live, code[1], sb[1]);
      store_row<D>(c, slot, head, live, code, sb);
    }
  }
}

// Read-back (kv_mxfp4_gather): the write's mapping reversed.
template <int D>
__global__ void __launch_bounds__(256) kv_gather_kernel(const KvView c, const int32_t* __restrict__ slots, int N,
                                                        uint4* __restrict__ ko, uint4* __restrict__ vo) {
  constexpr int L = D / 8, NB = D / 32;
  const long long rows = (long long)N * c.heads;
  const int sub = threadIdx.x % L, b = sub >> 2, t4 = sub & 3;
  const long long step = (long long)gridDim.x * (256 / L), first = (long long)blockIdx.x * (256 / L);
  RowWalk at(first + threadIdx.x / L, step, c.heads);
  for (long long w0 = first; w0 < rows; w0 += step * kRowsInFlight) {
    uint32_t code[kRowsInFlight][2], sb[kRowsInFlight][2];
    bool live[kRowsInFlight];
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
      const int head = at.head, slot = w0 + i * step + threadIdx.x / L < rows ? slots[at.tok] : -1;
      at.next();
      live[i] = slot >= 0 && (slot >> c.page_shift) < c.num_pages;
      code[i][0] = code[i][1] = sb[i][0] = sb[i][1] = 0u;
      if (live[i]) {
        const int off = slot & ((1 << c.page_shift) - 1), t = off & 15;
        const uint8_t* rec = c.data + c.record(slot >> c.page_shift, head, off >> 4);
        code[i][0] = *reinterpret_cast<const uint32_t*>(rec + k_byte<D>(t, 4 * sub));
        code[i][1] = *reinterpret_cast<const uint32_t*>(rec + v_byte<D>(t, 4 * t4 + 2 * (b & 1) + 16 * (b & ~1)));
        sb[i][0] = rec[16 * D + t * NB + b];
        sb[i][1] = rec[16 * D + D / 2 + t * NB + b];
      }
    }
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
      if (w0 + i * step >= rows) break;  // (uniform per CTA)
      const long long row = w0 + i * step + threadIdx.x / L;
      const uint32_t theirs = __shfl_xor_sync(0xffffffffu, code[i][1], 4);
      // even b: lower halves of b and b + 1; odd b: upper halves of b - 1 and b
      code[i][1] = (b & 1) ? prmt(theirs, code[i][1], 0x7632u) : prmt(code[i][1], theirs, 0x5410u);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t s = sb[i][w];
        // 2^(s-127) twice in bf16 (0: subnormal; 255: NaN); values and products are exact
        const uint32_t x = s == 0u ? 0x00400040u : s == 255u ? 0x7FFF7FFFu : s * 0x00800080u;
        uint32_t h[4], o[4];
        e2m1x8_to_f16x8(code[i][w], h[0], h[1], h[2], h[3]);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          o[q] = live[i] ? mul_bf16x2(prmt(__float_as_uint(f16_lo(h[q])), __float_as_uint(f16_hi(h[q])), 0x7632u), x) : 0u;
        if (row < rows) __stcs((w ? vo : ko) + row * L + sub, make_uint4(o[0], o[1], o[2], o[3]));
      }
    }
  }
}

int grid_for(long long units, int per_cta, int num_sms, int ctas_per_sm) {
  const long long want = (units + per_cta - 1) / per_cta, most = (long long)num_sms * ctas_per_sm;
  return (int)(want < most ? want : most);
}

}  // namespace

cudaError_t launch_page_tables(const PageTableArgs& a, int num_sms, cudaStream_t s) {
  const size_t smem = 4 * (3 * (size_t)a.R + 1);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(page_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               4 * (3 * kMaxTableRequests + 1));
    if (e != cudaSuccess) return e;
  }
  int grid = grid_for(a.max_tokens, kTableThreads, num_sms, 1);
  if (grid < 1) grid = 1;
  page_tables_kernel<<<grid, kTableThreads, smem, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_append(const KvView& c, const void* k, const void* v, bool f32, long long ks, long long vs, int N,
                             const int32_t* slots, int num_sms, cudaStream_t s) {
  const int grid = grid_for((long long)N * c.heads, 256 / (c.D / 8), num_sms, kRowCtas);
  if (c.D == 128) {
    if (f32) kv_append_kernel<128, true><<<grid, 256, 0, s>>>(c, k, v, ks, vs, N, slots);
    else kv_append_kernel<128, false><<<grid, 256, 0, s>>>(c, k, v, ks, vs, N, slots);
  } else {
    if (f32) kv_append_kernel<64, true><<<grid, 256, 0, s>>>(c, k, v, ks, vs, N, slots);
    else kv_append_kernel<64, false><<<grid, 256, 0, s>>>(c, k, v, ks, vs, N, slots);
  }
  return cudaGetLastError();
}

cudaError_t launch_kv_append_rope(const KvView& c, const RopeArgs& a, bool f32, bool pairs, int num_sms, cudaStream_t s) {
  const int W = 256 / c.D;  // units a warp
  const long long q_units = (long long)a.N * ((a.Hq + kQueryRows - 1) / kQueryRows), kv_units = (long long)a.N * c.heads;
  // one wave of resident warps, dealt to both kinds by their number of units (written and read
  // back, 16,384 tokens of 28 / 4 heads of 128: 3 CTAs an SM 57.7 us, 8, not all resident, 63.8)
  const long long most = (long long)num_sms * rope_ctas(f32) * 8;
  long long qw = (q_units + W - 1) / W, kw = (kv_units + W - 1) / W;
  if (qw + kw > most) {
    const long long share = std::max<long long>(1, most * qw / (qw + kw));
    qw = qw ? std::min(share, most - 1) : 0;
    kw = most - qw;
  }
  const int grid = (int)((qw + kw + 7) / 8);
  auto go = [&](auto d, auto wide, auto p) {
    kv_append_rope_kernel<decltype(d)::value, decltype(wide)::value, decltype(p)::value><<<grid, 256, 0, s>>>(c, a, (int)qw);
  };
  auto of_dim = [&](auto wide, auto p) {
    if (c.D == 128) go(std::integral_constant<int, 128>{}, wide, p);
    else go(std::integral_constant<int, 64>{}, wide, p);
  };
  auto of_type = [&](auto p) {
    if (f32) of_dim(std::true_type{}, p);
    else of_dim(std::false_type{}, p);
  };
  if (pairs) of_type(std::true_type{});
  else of_type(std::false_type{});
  return cudaGetLastError();
}

cudaError_t launch_kv_gather(const KvView& c, const int32_t* slots, int N, void* ko, void* vo, int num_sms,
                             cudaStream_t s) {
  const int grid = grid_for((long long)N * c.heads, 256 / (c.D / 8), num_sms, kRowCtas);
  if (c.D == 128)
    kv_gather_kernel<128><<<grid, 256, 0, s>>>(c, slots, N, reinterpret_cast<uint4*>(ko), reinterpret_cast<uint4*>(vo));
  else
    kv_gather_kernel<64><<<grid, 256, 0, s>>>(c, slots, N, reinterpret_cast<uint4*>(ko), reinterpret_cast<uint4*>(vo));
  return cudaGetLastError();
}

}  // namespace moe
