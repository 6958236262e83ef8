// The 4-bit KV cache outside attention: page tables and slot maps from request
// lengths, the quantising write of new rows, and the read-back.
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

// Quantising write (kv_mxfp4_append).  HBM-bound: 2 or 4 bytes read and 17/32
// byte written per value (16,384 x 8 x 128, written and read back: 31.4 us, 5.4
// TB/s of the bytes that both must move).  D / 8 lanes take a token's K and V row of one head;
// the loop bounds are uniform per warp, so every lane reaches the shuffles.
// Neighbouring blocks' lanes trade halves of their V words, so that each writes
// four bytes of one lane's operand.
template <int D, bool F32>
__global__ void __launch_bounds__(256) kv_append_kernel(const KvView c, const void* __restrict__ k,
                                                        const void* __restrict__ v, long long ks, long long vs, int N,
                                                        const int32_t* __restrict__ slots) {
  constexpr int L = D / 8, NB = D / 32;  // lanes per row
  const long long rows = (long long)N * c.heads;
  const int sub = threadIdx.x % L, b = sub >> 2, t4 = sub & 3;
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
      // V: lanes of blocks b and b ^ 1 hold bytes 2 t4 (lower half) and 2 t4 + 1
      // (upper) of their blocks; even b takes the lower halves of both, odd b the upper
      const uint32_t theirs = __shfl_xor_sync(0xffffffffu, code[1], 4);
      const uint32_t vw = (b & 1) ? prmt(theirs, code[1], 0x7632u) : prmt(code[1], theirs, 0x5410u);
      if (live) {
        const int off = slot[i] & ((1 << c.page_shift) - 1), t = off & 15;
        uint8_t* rec = c.data + c.record(slot[i] >> c.page_shift, head[i], off >> 4);
        *reinterpret_cast<uint32_t*>(rec + k_byte<D>(t, 4 * sub)) = code[0];
        *reinterpret_cast<uint32_t*>(rec + v_byte<D>(t, 4 * t4 + 2 * (b & 1) + 16 * (b & ~1))) = vw;
        if (t4 < 2) rec[16 * D + t4 * (D / 2) + t * NB + b] = (uint8_t)sb[t4];
      }
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
