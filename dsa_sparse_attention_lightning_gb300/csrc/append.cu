// append.cu -- new tokens from raw projections into the paged caches: RMS norm
// of the 512 compressed dims, rotation of the 64 RoPE dims, quantization and the
// paged write in one pass, with the index key of the Write step beside it.
//
// Per new token t (x = latent[t], 576 values):
//   c[d] = gamma[d] * x[d] / sqrt(mean_{d < 512} x[d]^2 + eps)        (d < 512)
//   r    = mscale * R(tok_pos[t]) x[512:576], pairs (2i, 2i + 1) or (i, i + 32)
// then E4M3(v / latent_scale) of all 576 values (FP8 rows), or (NVFP4 rows) per
// block of 16 of the first 512, v = c / latent_scale:
//   s = E4M3(max |v| / 6), codes E2M1(v / s) (0 where s is 0), and E4M3(r / latent_scale).
// The values stay in fp32 registers from the load to the one rounding into the
// cache; the sum of squares is an fp32 warp reduction.
//
// One warp per token: lane l holds dims 8l .. 8l + 7 and 256 + 8l .. (two 16-byte loads, each
// of the warp 512 contiguous bytes; two lanes an NVFP4 block) and RoPE pair l.  Every load of
// a token but its page number is issued before any is used, and the page number is waited for
// behind the norm and the rotation.  CTAs of four warps, at most eight per SM (a warp takes
// several tokens then), and no variant may have more than the 64 registers that this leaves: with 72 and
// seven CTAs 100000 tokens with FP8 keys and NVFP4 rows take 91 us instead of 72, with MXFP4 keys and
// FP8 rows 78 instead of 64.
// Measured, inputs not in L2: 64 tokens with FP8 keys and rows 2.7 us, 4096 with MXFP4 keys and NVFP4
// rows 5.1, 16383 latent rows 8.7, 100000 37.5 (4.6 TB/s); with FP8 keys 57.6, with MXFP4 keys and NVFP4
// rows 78.  A CTA for every four tokens, 16 consecutive dims per lane, kept values, looked-up pages
// and fewer registers for more warps were slower (16383 rows of inputs in L2: 7.6, 8.1, 7.3 and 6.5
// instead of 6.3; 9.3 cold); rows prefetched by cp.async gain 7 % without an index key and lose 4 % with one.
#include "dsa_common.cuh"
#include "rope_common.cuh"
#include "write_common.cuh"

namespace dsa {
namespace {

constexpr int kAppWarps = 4;
constexpr int kAppCtasPerSm = 8;
constexpr int kNvCodeBytes = 256, kNvScaleBytes = 32, kNvRow = 352;
enum { kNoKey = 0, kFp8Key = 1, kMxKey = 2 };

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Eight floats -> eight E2M1 codes (round to nearest even, beyond 6 clamped),
// the first in the low nibble of byte 0.
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// x / d rounded to nearest, from rd = 1 / d rounded to nearest: one correction of the product by its
// exact remainder (P. Markstein, IBM J. Res. Dev. 34, 1990), which is taken negative so that 0 keeps
// its sign.  Infinities and NaN are the product's.
__device__ __forceinline__ float quotient(float x, float d, float rd) {
  const float q = x * rd, c = fmaf(-fmaf(q, d, -x), rd, q);
  return fabsf(q) < INFINITY ? c : q;
}

__device__ __forceinline__ float bf16_val(const uint16_t* p) {
  return __uint_as_float((uint32_t)*p << 16);
}

template <int kKey, bool kNv>
__global__ void __launch_bounds__(kAppWarps * 32, kAppCtasPerSm)
append_kv_kernel(const uint16_t* __restrict__ latent, int64_t lat_row,
                 const float* __restrict__ lat_gamma, float lat_eps,
                 const double* __restrict__ inv_freq, float mscale, int interleaved,
                 float latent_scale, float inv_scale, const uint16_t* __restrict__ k_raw, int64_t k_row,
                 const float* __restrict__ key_gamma, const float* __restrict__ key_beta,
                 float key_eps, const int32_t* __restrict__ block_table, int B, int max_pages,
                 const int32_t* __restrict__ tok_req, const int32_t* __restrict__ tok_pos, int T,
                 uint8_t* __restrict__ key_cache, uint8_t* __restrict__ latent_cache,
                 int64_t num_pages, uint32_t* status) {
  const int lane = threadIdx.x & 31;
  const int ra = interleaved ? 2 * lane : lane, rb = interleaved ? 2 * lane + 1 : lane + 32;
  uint64_t fraction = 0;
  bool fresh = true;
  for (int64_t t = (int64_t)blockIdx.x * kAppWarps + (threadIdx.x >> 5); t < T;
       t += (int64_t)gridDim.x * kAppWarps) {
    const int req = tok_req[t], pos = tok_pos[t];
    const uint16_t* x = latent + t * lat_row;
    const uint4 wa = reinterpret_cast<const uint4*>(x)[lane];
    const uint4 wb = reinterpret_cast<const uint4*>(x)[lane + 32];
    const float xa = bf16_val(x + kVDim + ra), xb = bf16_val(x + kVDim + rb);
    KeyIn key;
    if constexpr (kKey != kNoKey) key = load_index_key(k_raw + t * k_row, key_gamma, key_beta, lane);
    if (inv_freq && fresh) fraction = turn_fraction(inv_freq[lane]);
    fresh = false;
    if (pos == -1) continue;                            // padding
    if (req < 0 || req >= B || pos < 0 || (int64_t)pos >= (int64_t)max_pages * kPage) {
      if (lane == 0) raise_dev(status, DSA_DEV_BAD_ROW);
      continue;
    }
    const int page = block_table[(size_t)req * max_pages + pos / kPage];
    // while the page number is on its way: the norm and the rotation
    const uint32_t w[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
    float v[16];
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
      sq = fmaf(v[2 * i], v[2 * i], fmaf(v[2 * i + 1], v[2 * i + 1], sq));
    }
    if (lat_gamma) {
      const float f = inv_scale * rsqrtf(warp_sum(sq) / (float)kVDim + lat_eps);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 g = reinterpret_cast<const float4*>(lat_gamma + 256 * (i >> 1))[2 * lane + (i & 1)];
        v[4 * i] *= f * g.x; v[4 * i + 1] *= f * g.y; v[4 * i + 2] *= f * g.z; v[4 * i + 3] *= f * g.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = quotient(v[i], latent_scale, inv_scale);   // as dsa_write_kv
    }
    float2 r = make_float2(xa, xb);
    if (inv_freq) r = rotate(xa, xb, rotation(fraction, pos, mscale));
    const uint32_t rr = pack_e4m3x4(quotient(r.x, latent_scale, inv_scale),
                                    quotient(r.y, latent_scale, inv_scale), 0.f, 0.f);
    if (page < 0 || (int64_t)page >= num_pages) {
      if (lane == 0) raise_dev(status, DSA_DEV_BAD_PAGE);
      continue;
    }
    const int slot = pos % kPage;
    if constexpr (kKey != kNoKey)
      write_index_key<kKey == kMxKey>(key, key_eps, key_cache, page, slot, lane);
    uint8_t* row = latent_cache + ((size_t)page * kPage + slot) * (kNv ? kNvRow : kLatDim);
    uint8_t* rope = row + (kNv ? kNvCodeBytes + kNvScaleBytes : kVDim);
    if constexpr (kNv) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {                   // dims 256 h + 8 lane ..: half of block 16 h + lane / 2
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max_nan(amax, fabsf(v[8 * h + i]));
        amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        const uint8_t sb = __nv_cvt_float_to_fp8(amax / 6.f, __NV_SATFINITE, __NV_E4M3);
        const float s = e4m3_to_float(sb);
        const float is = s > 0.f ? 1.f / s : 0.f;
        // quotients: the product with 1 / s would move values off the middle between two codes.  Divisions
        // take 5.4 us for 4096 tokens (in L2, with FP4 keys), these 5.0, products 4.9
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * h + i] = quotient(v[8 * h + i], s, is);
        // (a negative value times 0 would be the code of -0)
        reinterpret_cast<uint32_t*>(row)[32 * h + lane] = is > 0.f ? e2m1x8(v + 8 * h) : 0;
        if (lane % 2 == 0) row[kNvCodeBytes + 16 * h + lane / 2] = sb;
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        reinterpret_cast<uint2*>(row)[32 * h + lane] =
            make_uint2(pack_e4m3x4(v[8 * h], v[8 * h + 1], v[8 * h + 2], v[8 * h + 3]),
                       pack_e4m3x4(v[8 * h + 4], v[8 * h + 5], v[8 * h + 6], v[8 * h + 7]));
    }
    if (interleaved) {
      reinterpret_cast<uint16_t*>(rope)[lane] = (uint16_t)rr;
    } else {
      rope[ra] = (uint8_t)rr;
      rope[rb] = (uint8_t)(rr >> 8);
    }
  }
}

}  // namespace

cudaError_t launch_append_kv(const AppendArgs& a, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  const int need = (a.T + kAppWarps - 1) / kAppWarps;
  const int grid = need < kMlaGrid * kAppCtasPerSm ? need : kMlaGrid * kAppCtasPerSm;
  auto go = [&](auto kernel) {
    kernel<<<grid, kAppWarps * 32, 0, st>>>(
        static_cast<const uint16_t*>(a.latent), a.lat_row, a.lat_gamma, a.lat_eps, a.inv_freq,
        a.mscale, a.interleaved ? 1 : 0, a.latent_scale, 1.f / a.latent_scale,
        static_cast<const uint16_t*>(a.k_raw), a.k_row, a.key_gamma, a.key_beta, a.key_eps,
        a.block_table, a.B, a.max_pages, a.tok_req, a.tok_pos, a.T, a.key_cache, a.latent_cache,
        a.num_pages, a.status);
  };
  if (a.nvfp4) {
    if (!a.key_cache) go(append_kv_kernel<kNoKey, true>);
    else if (a.mx_keys) go(append_kv_kernel<kMxKey, true>);
    else go(append_kv_kernel<kFp8Key, true>);
  } else {
    if (!a.key_cache) go(append_kv_kernel<kNoKey, false>);
    else if (a.mx_keys) go(append_kv_kernel<kMxKey, false>);
    else go(append_kv_kernel<kFp8Key, false>);
  }
  return cudaGetLastError();
}

}  // namespace dsa
