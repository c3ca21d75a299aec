// weights_share.cuh — how the tcgen05 kernel of the collected attention weight deals its key tiles to the CTAs (internal to
// libfpd; host code too, so that the deal is tested without a GPU).
#pragma once

#include "fpd_internal.cuh"

namespace fpd {

constexpr int kShareTile = 128;   // keys of a tile

// The key tiles of one CTA: an even run of all (request, kv head, key tile) that hold a key, requests in order.  len(b): request
// b's length.  Lengths that another stream changes meanwhile may deal the tiles wrongly, but every walk ends and stays within
// the requests.
template <class Len>
struct Share {
  Len len;
  int batch, nkv;
  int b, g, kt, tiles, T;   // request, kv head, next tile, the request's tiles and length
  long long left;
  int nk, k0;               // unit: nk key tiles of one request and kv head, the first at key k0

  __host__ __device__ static int tiles_of(int n) { return n / kShareTile + (n % kShareTile != 0); }
  __host__ __device__ void load(int b_) {
    b = b_;
    T = b < batch ? len(b) : 0;
    tiles = tiles_of(T);
  }
  __host__ __device__ long long count(int i) { return i < batch ? (long long)nkv * tiles_of(len(i)) : 0ll; }
  __host__ __device__ long long count32(int i0) {   // tiles of requests i0 .. i0 + 31; by a whole warp
#ifdef __CUDA_ARCH__
    long long v = count(i0 + (threadIdx.x & 31));
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
#else
    long long v = 0;
    for (int i = 0; i < 32; i++) v += count(i0 + i);
#endif
    return v;
  }
  __host__ __device__ Share(Len len_, int batch_, int nkv_, int cta, int ctas) : len(len_), batch(batch_), nkv(nkv_) {
    long long total = 0;
    for (int i0 = 0; i0 < batch; i0 += 32) total += count32(i0);
    long long lo = cta * total / ctas;
    left = (cta + 1) * total / ctas - lo;
    int i0 = 0;
    for (; left > 0 && i0 < batch; i0 += 32) {   // the 32 requests, then the request, that hold tile lo
      const long long c = count32(i0);
      if (lo < c) break;
      lo -= c;
    }
    load(i0);
    while (left > 0 && b < batch && lo >= (long long)nkv * tiles) {
      lo -= (long long)nkv * tiles;
      load(b + 1);
    }
    if (b >= batch) left = 0;
    g = left > 0 ? (int)(lo / tiles) : 0;
    kt = left > 0 ? (int)(lo - (long long)g * tiles) : 0;
    nk = 0;
  }
  __host__ __device__ bool next() {
    kt += nk;
    left -= nk;
    nk = 0;
    if (left <= 0) return false;
    while (kt >= tiles) {
      kt = 0;
      if (++g >= nkv || tiles == 0) {
        g = 0;
        if (b + 1 >= batch) {
          left = 0;
          return false;
        }
        load(b + 1);
      }
    }
    k0 = kt * kShareTile;
    nk = tiles - kt < 2 || left < 2 ? 1 : 2;
    return true;
  }
};

}  // namespace fpd
