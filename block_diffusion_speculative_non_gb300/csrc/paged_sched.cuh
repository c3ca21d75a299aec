// paged_sched.cuh — how the key tiles of a paged attention call are shared out (internal to libfpd).
//
// A unit is a row tile of one request and kv head: rows (position, head) rt R .. of the L positions' heads that share the kv
// head.  It has the key tiles that hold a key some row of it sees: those of the first `sinks` positions, those from the first
// row's window to the end, then the block's keys.  The lengths are known on the device alone, and requests differ in them, so
// every CTA adds them up and takes an even run of all units' tiles (the first runs one tile more than the others): whatever the
// lengths, the SMs finish together.  A unit also counts for what it costs besides its tiles (its queries, its way out).  A unit inside one run is
// finished there; of a unit that runs share, each leaves a partial: the run
// that starts it in slot 2 c + 1, the ones that go on with it in slot 2 c.  A unit without a key counts as one empty tile, so
// that its rows are written too.
#pragma once

#include "fpd_paged.cuh"

namespace fpd {

constexpr int kPagedTile = 64, kPagedTcTile = 128;   // keys of a tile of k_paged_stream.cu and of k_paged_tc.cu
constexpr int kSchedEntries = 32;    // the lanes of a warp add up ceil(batch / 32) requests each

struct PagedUnit {
  int b, g, rt;
  int T, n, p0, p1;          // context length, keys, positions of the tile's first and last row
  int ce, be;                // context slots and block keys before the end of what the rows see
  int ns, cfirst, nm;        // tiles of the sinks; first tile behind them and their number
  int bfirst, nb;            // first tile of the block and their number
  __host__ __device__ int tiles() const { return ns + nm + nb; }
  __host__ __device__ int len() const { return tiles() > 0 ? tiles() : 1; }
};

struct PagedTile {
  bool ctx;
  int k0, valid, pos;   // first slot or block key, keys, position of the first
};

__host__ __device__ inline int imin(int a, int b) { return a < b ? a : b; }
__host__ __device__ inline int imax(int a, int b) { return a > b ? a : b; }

// Division of 0 <= x < 2^31 by a number known on the host (Granlund and Montgomery's multiply, add and shift): the walk divides by
// the group several times a unit, and the compiler's division by a variable is some 30 instructions.
struct GroupDiv {
  uint32_t d, m, s1, s2;
  void set(uint32_t n) {
    d = n;
    uint32_t l = 0;
    while ((1ull << l) < n) l++;
    m = (uint32_t)(((1ull << 32) * ((1ull << l) - n)) / n + 1);
    s1 = l > 0 ? 1 : 0;
    s2 = l > 0 ? l - 1 : 0;
  }
  __host__ __device__ int div(int x) const {
#ifdef __CUDA_ARCH__
    const uint32_t t = __umulhi(m, (uint32_t)x);
#else
    const uint32_t t = (uint32_t)(((uint64_t)m * (uint32_t)x) >> 32);
#endif
    return (int)((t + (((uint32_t)x - t) >> s1)) >> s2);
  }
};

// What decides a unit's tiles.
struct PagedShape {
  int L, lb, grp, nkv, rows, tiles, window, sinks, causal;   // rows of a row tile, row tiles of a request and kv head
  int kt_shift;                                              // tiles of 2^kt_shift keys
  int unit_cost;                                             // what a unit costs besides its tiles, in tiles
  GroupDiv by_grp;
  __host__ __device__ int kt() const { return 1 << kt_shift; }
};
inline PagedShape paged_shape(int L, int lb, int grp, int nkv, int rows, int window, int sinks, int causal, int kt,
                              int unit_cost) {
  PagedShape s{L, lb, grp, nkv, rows, ceil_div(L * grp, rows), window, sinks, causal, 0, unit_cost, {}};
  while (s.kt() < kt) s.kt_shift++;
  s.by_grp.set(grp);
  return s;
}

__host__ __device__ inline void unit_tiles(const PagedShape& s, int T, int rt, PagedUnit& u) {
  const int sh = s.kt_shift, up = s.kt() - 1;
  u.rt = rt;
  u.T = T;
  u.n = T + s.lb;
  const int last = imin(s.L * s.grp, (rt + 1) * s.rows) - 1;
  u.p0 = u.n - s.L + s.by_grp.div(rt * s.rows);
  u.p1 = u.n - s.L + s.by_grp.div(last);
  const int end = s.causal ? imin(u.n, imax(0, u.p1 + 1)) : u.n;
  const int start = s.window ? imin(end, imax(0, u.p0 - s.window + 1)) : 0;
  const int s_end = imin(s.sinks, start);
  u.ce = imin(end, T);
  u.be = imax(0, end - T);
  u.ns = (imin(s_end, u.ce) + up) >> sh;
  u.cfirst = imax(start >> sh, u.ns);
  u.nm = start < u.ce ? imax(0, ((u.ce + up) >> sh) - u.cfirst) : 0;
  u.bfirst = s_end > T ? 0 : imax(0, start - T) >> sh;
  u.nb = imax(0, ((u.be + up) >> sh) - u.bfirst);
}

__host__ __device__ inline PagedTile tile_at(const PagedUnit& u, int kt, int i) {
  PagedTile t;
  t.ctx = i < u.ns + u.nm;
  const int idx = i < u.ns ? i : t.ctx ? u.cfirst + i - u.ns : u.bfirst + i - u.ns - u.nm;
  t.k0 = idx * kt;
  t.valid = imin(kt, (t.ctx ? u.ce : u.be) - t.k0);
  t.pos = t.ctx ? t.k0 : u.T + t.k0;
  return t;
}
// Whether every row of the unit sees every key of the tile.
__host__ __device__ inline bool tile_full(const PagedShape& s, const PagedUnit& u, const PagedTile& t) {
  const int last = t.pos + s.kt() - 1;
  return t.valid == s.kt() && (!s.window || last < s.sinks || u.p1 - t.pos < s.window) && (!s.causal || last <= u.p0);
}

// Tiles of a request in one kv head, with what its units cost besides.
__host__ __device__ inline int request_tiles(const PagedShape& s, int T) {
  PagedUnit u;
  if (!s.window && !s.causal) {
    unit_tiles(s, T, 0, u);
    return s.tiles * (u.len() + s.unit_cost);
  }
  int n = 0;
  for (int rt = 0; rt < s.tiles; rt++) {
    unit_tiles(s, T, rt, u);
    n += u.len() + s.unit_cost;
  }
  return n;
}

// One run over the units.  Lens: the length of request b, clamped.  The host sees to it that all tiles fit 31 bits.
template <class Lens>
struct PagedWalk {
  const PagedShape& s;
  Lens lens;
  int c, G, batch, b, g, rt, off;
  int x, x_end, each_run, longer;   // runs of each_run tiles, the first `longer` of them one more

  __host__ __device__ PagedWalk(const PagedShape& s_, Lens lens_, int batch_, int total, int runs, int c_)
      : s(s_), lens(lens_), c(c_), batch(batch_), b(0), g(0), rt(0), off(0) {
    G = imin(total, runs);
    each_run = (int)((unsigned)total / (unsigned)G);
    longer = total - each_run * G;
    x = c < G ? run_start(c) : total;
    x_end = c < G ? run_start(c + 1) : total;
  }
  // Finds the run's first unit: entry lo, which starts at tile `base` and holds `size` of them, is the one with tile x.
  __host__ __device__ void locate(int lo, int base, int size) {
    const int each = (batch + kSchedEntries - 1) / kSchedEntries;
    int rest = x - base, per;
    b = lo * each;
    if (each == 1) {
      per = (int)((unsigned)size / (unsigned)s.nkv);
    } else {
      for (;; b++) {
        per = request_tiles(s, lens(b));
        if (rest < per * s.nkv || b + 1 >= batch) break;
        rest -= per * s.nkv;
      }
    }
    // lengths that another stream changes meanwhile give a wrong result, never a unit that is not there
    g = imin((int)((unsigned)rest / (unsigned)per), s.nkv - 1);
    rest -= g * per;
    PagedUnit u;
    if (!s.window && !s.causal) {
      unit_tiles(s, lens(b), 0, u);
      rt = imin((int)((unsigned)rest / (unsigned)(u.len() + s.unit_cost)), s.tiles - 1);
      rest -= rt * (u.len() + s.unit_cost);
    } else {
      for (rt = 0; rt + 1 < s.tiles; rt++) {
        unit_tiles(s, lens(b), rt, u);
        if (rest < u.len() + s.unit_cost) break;
        rest -= u.len() + s.unit_cost;
      }
      unit_tiles(s, lens(b), rt, u);
    }
    off = rest;
    if (off >= u.len()) {   // among what the unit costs besides: the run starts with the next one
      x += imax(1, u.len() + s.unit_cost - off);
      step();
    }
  }
  __host__ __device__ void step() {   // to the next unit
    off = 0;
    if (++rt == s.tiles) {
      rt = 0;
      if (++g == s.nkv) {
        g = 0;
        b++;
      }
    }
  }
  __host__ __device__ int run_start(int i) const { return i * each_run + imin(i, longer); }
  __host__ __device__ int run_of(int t) const {
    const int before = longer * (each_run + 1);   // tiles of the longer runs
    return (int)(t < before ? (unsigned)t / (unsigned)(each_run + 1) : longer + (unsigned)(t - before) / (unsigned)each_run);
  }

  // The next part [t0, t1) of a unit's tiles; last_run: the run that ends the unit.
  __host__ __device__ bool next(PagedUnit& u, int& t0, int& t1, int& last_run) {
    if (x >= x_end || b >= batch) return false;
    unit_tiles(s, lens(b), rt, u);
    u.b = b;
    u.g = g;
    const int len = u.len();
    if (off >= len) off = len - 1;
    t0 = off;
    t1 = imin(len, off + (x_end - x));
    if (t1 == len) {
      last_run = c;
      x += len + s.unit_cost - off;
      step();
    } else {
      last_run = imin(run_of(x + (len - off) - 1), G - 1);
      x = x_end;
    }
    return true;
  }
};

cudaError_t paged_stream_init_attributes();
int paged_stream_warps(int rows, int format);   // runs per SM
// per_cta: a CTA for each unit, which leaves no partial
cudaError_t launch_paged_stream(const PagedAttn& a, const PagedShape& s, const PagedPlan& pl, bool per_cta, cudaStream_t st);

cudaError_t paged_tc_init_attributes();
cudaError_t launch_paged_tc(const PagedAttn& a, const PagedShape& s, const PagedPlan& pl, cudaStream_t st);

#ifdef __CUDACC__
struct DeviceLens {
  const int32_t* ctx_len;
  int cap;
  __device__ int operator()(int b) const { return clamp_ctx(ctx_len[b], cap); }
};
// The walk of run c, by a whole warp (every warp that walks makes its own; no shared memory, no barrier).
__device__ __forceinline__ PagedWalk<DeviceLens> make_walk(const PagedShape& s, DeviceLens lens, int batch, int runs, int c) {
  const int each = (batch + kSchedEntries - 1) / kSchedEntries, lane = threadIdx.x & 31;
  int v = 0;
  for (int b = lane * each; b < min(batch, (lane + 1) * each); b++) v += s.nkv * request_tiles(s, lens(b));
  int up = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += t;
  }
  PagedWalk<DeviceLens> w(s, lens, batch, __shfl_sync(0xffffffffu, up, 31), runs, c);
  const unsigned m = __ballot_sync(0xffffffffu, up > w.x);
  const int e = m ? __ffs(m) - 1 : 31;
  const int base = __shfl_sync(0xffffffffu, up - v, e), size = __shfl_sync(0xffffffffu, v, e);
  if (w.x < w.x_end) w.locate(e, base, size);
  return w;
}
#endif

}  // namespace fpd
