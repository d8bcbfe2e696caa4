// Shared prefixes: how the SMs are dealt between the kernel over the prefixes and the decodes of the sequences' own
// tokens beside it (prefill.cu, shared_prefix.cu).
#pragma once

#include <math.h>
#include <string.h>

namespace metis {

// How many of the grid's CTAs (one per SM) share the prefixes' K/V tiles, so that these and the decodes of the
// sequences' own tokens, on the other SMs at the same time, end together.  A CTA takes 7 us to
// start, 5 us for each unit (its queries, its parts) and 2 us a tile; decodes of own tokens stream 40 GB/s on each of
// their SMs, 6.1 TB/s together.  These figures were fitted at two batches: 64 sequences behind 16,384 tokens (8 units)
// take 64 CTAs, 52.3 us; 1,024 behind 16 prompts of about 600 (256 units) 26, 110 us (the own tokens behind the
// prefixes, each on all SMs: 58.9 and 129).  Between them, 8 groups of 32 behind 2,048 tokens (64 units): 82.7 us.
constexpr float kShareStartUs = 7.f, kShareUnitUs = 5.f, kShareTileUs = 2.f;
constexpr float kOwnBytesPerUs = 40e3f, kOwnBytesPerUsAll = 6.1e6f;

// What n of `sms` CTAs would take, in whole sixteenths of a microsecond (the bits of that fp32, which order as its
// values do and do not saturate), above n itself: the smallest key's n is the one to take.
__host__ __device__ __forceinline__ unsigned long long shared_split_key(int tiles, int units, float own_bytes, int n,
                                                                        int sms) {
  const float prefix = kShareStartUs + kShareTileUs * (((unsigned)tiles + n - 1) / n) +
                       kShareUnitUs * (((unsigned)units + n - 1) / n);
  const float rate = kOwnBytesPerUs * (sms - n) < kOwnBytesPerUsAll ? kOwnBytesPerUs * (sms - n) : kOwnBytesPerUsAll;
  const float own = n < sms ? kShareStartUs + own_bytes / rate : 0.f;
  const float sixteenths = floorf(16.f * (prefix > own ? prefix : own));
  unsigned bits;
  memcpy(&bits, &sixteenths, 4);
  return (unsigned long long)bits << 32 | (unsigned)n;
}

// The counts to choose from: 1 .. this (an SM at least for own tokens)
__host__ __device__ __forceinline__ int shared_split_most(float own_bytes, int sms) {
  return own_bytes > 0.f && sms > 1 ? sms - 1 : sms;
}

}  // namespace metis
