// paged_repair.cuh — what becomes of values that are not finite where a mask hides them (internal to libfpd).
//
// A product takes weight 0 times such a value to NaN.  V rows that no row of a unit sees are zeroed before their product; a
// value that some rows see and others do not (in the window's first tiles, in a causal block) spoils the others.  So where masks
// differ between rows and a row's O came out without a number, that row's O is summed once more, over the keys it sees and
// none else.  A row that does see such a value comes out as it should, and soon: the sum ends when no dim holds a number.
#pragma once

#include "paged_sched.cuh"

namespace fpd {

__device__ __forceinline__ bool row_sees(const PagedShape& s, int row, int pos) {
  return (!s.window || pos < s.sinks || row - pos < s.window) && (!s.causal || pos <= row);
}

// Keys [lo, hi) of a tile that a window hides from every row of the unit.
__device__ __forceinline__ void hidden_from_all(const PagedShape& s, const PagedUnit& u, const PagedTile& t, int& lo, int& hi) {
  lo = hi = 0;
  if (!s.window) return;
  lo = max(0, s.sinks - t.pos);
  hi = max(lo, min(t.valid, u.p0 - s.window + 1 - t.pos));
}

// Row `pos` (null: zeros) of K or V of a tile's key k.
template <int H>
struct KeyRow {
  const bf16* plain = nullptr;
  const uint8_t *code = nullptr, *scale = nullptr;
  __device__ __forceinline__ void locate(const PagedAttn& a, const PagedUnit& u, const PagedTile& t, int k, int is_v) {
    if (!t.ctx) {
      plain = (is_v ? a.vblk : a.kblk) + (((size_t)u.b * a.pg.nkv + u.g) * a.lb + t.k0 + k) * H;
      return;
    }
    const int slot = t.k0 + k, id = page_of(a.pg, u.b, slot), in = slot & (a.pg.page - 1);
    if (id < 0) return;
    const uint8_t* slab = slab_of(a.pg, id, is_v, u.g);
    if (a.pg.format == FPD_PAGE_BF16) {
      plain = reinterpret_cast<const bf16*>(slab) + (size_t)in * H;
    } else {
      code = slab + in * (H / 2);
      scale = slab + a.pg.page * (H / 2) + in * (H / 16);
    }
  }
  __device__ __forceinline__ float at(int d) const {
    if (plain) return __bfloat162float(plain[d]);
    if (!code) return 0.f;
    return (float)((code[d >> 1] >> (4 * (d & 1)) & 15) - 8) * scale_value(scale[d >> 4]);
  }
};

// acc[j], dim lane + 32 j: sum over the keys of tiles [t0, t1) that the row sees of 2^(s log2(e) / sqrt(h) - m) v, by one warp.  qi: the
// row among the unit's request and kv head; m: the row's maximum in base 2.
template <int H>
__device__ __noinline__ void repair_row(const PagedAttn& a, const PagedShape& s, const PagedUnit u, int t0, int t1, int qi, float m,
                                        float (&acc)[H / 32]) {
  const int lane = threadIdx.x & 31, row = u.n - a.L + qi / s.grp;
  const bf16* q = a.q + ((size_t)(u.b * a.L + qi / s.grp) * a.nq + u.g * s.grp + qi % s.grp) * H;
  const float sl2 = rsqrtf((float)H) * 1.4426950408889634f;
#pragma unroll
  for (int j = 0; j < H / 32; j++) acc[j] = 0.f;
  for (int i = t0; i < t1; i++) {
    const PagedTile t = tile_at(u, s.kt(), i);
    for (int k0 = 0; k0 < t.valid; k0 += 32) {   // a key per lane, then the keys' values one after the other
      const int k = k0 + lane;
      const bool see = k < t.valid && row_sees(s, row, t.pos + k);
      float p = 0.f;
      if (see) {
        KeyRow<H> r;
        r.locate(a, u, t, k, 0);
        float dot = 0.f;
        for (int d = 0; d < H; d++) dot = fmaf(__bfloat162float(q[d]), r.at(d), dot);
        p = exp2f(fmaf(dot, sl2, -m));
      }
      unsigned left = __ballot_sync(0xffffffffu, see);
      while (left) {
        const int e = __ffs(left) - 1;
        left &= left - 1;
        const float w = __shfl_sync(0xffffffffu, p, e);
        KeyRow<H> r;
        r.locate(a, u, t, k0 + e, 1);
#pragma unroll
        for (int j = 0; j < H / 32; j++) acc[j] = fmaf(w, r.at(lane + 32 * j), acc[j]);
      }
      bool number = false;
#pragma unroll
      for (int j = 0; j < H / 32; j++) number |= acc[j] == acc[j];
      if (!__any_sync(0xffffffffu, number)) return;
    }
  }
}

}  // namespace fpd
