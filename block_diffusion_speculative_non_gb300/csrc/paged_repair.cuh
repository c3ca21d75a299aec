// paged_repair.cuh — what becomes of values that are not finite where a mask hides them (internal to libfpd).
//
// A product takes weight 0 times such a value to NaN.  V rows that no row of a unit sees are zeroed before their product; a
// value that some rows see and others do not (in the window's first tiles, in a causal block) spoils the others.  So where masks
// differ between rows and a row came out without a number, the merge sums that row once more, over the keys it sees and none
// else.  A row that does see such a value comes out as it should, and soon: the sum ends when no dim holds a number.
#pragma once

#include "paged_masks.cuh"

namespace fpd {

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

// acc[j], dim lane + 32 j: sum over the keys of the unit that the row sees of 2^(s log2(e) / sqrt(h) - m) v, by one warp, and `den`, the sum
// of the weights.  qi: the row among the request's and kv head's; m: the row's maximum in base 2, or NaN: it is taken first.
template <int H>
__device__ __noinline__ void repair_row(const PagedAttn& a, const PagedShape& s, const PagedUnit u, int qi, float m, float (&acc)[H / 32],
                                        float& den) {
  const int lane = threadIdx.x & 31, row = u.n - a.L + qi / s.grp;
  const bf16* q = a.q + ((size_t)(u.b * a.L + qi / s.grp) * a.nq + u.g * s.grp + qi % s.grp) * H;
  const float sl2 = rsqrtf((float)H) * 1.4426950408889634f;
  const bool find = m != m;
  if (find) m = -INFINITY;
  for (int pass = find ? 0 : 1; pass < 2; pass++) {
#pragma unroll
    for (int j = 0; j < H / 32; j++) acc[j] = 0.f;
    den = 0.f;
    for (int i = 0; i < u.tiles(); i++) {
      const PagedTile t = tile_at(u, s.kt(), i);
      for (int k0 = 0; k0 < t.valid; k0 += 32) {   // a key per lane, then the keys' values one after the other
        const int k = k0 + lane;
        const bool see = k < t.valid && row_sees(s, row, t.pos + k);
        float x = -INFINITY;
        if (see) {
          KeyRow<H> r;
          r.locate(a, u, t, k, 0);
          float dot = 0.f;
          for (int d = 0; d < H; d++) dot = fmaf(__bfloat162float(q[d]), r.at(d), dot);
          x = dot * sl2;
        }
        if (pass == 0) {
          m = fmaxf(m, warp_max(x));
          continue;
        }
        const float p = see ? exp2f(x - (m == -INFINITY ? 0.f : m)) : 0.f;
        den += warp_sum(p);
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
}

}  // namespace fpd
