// How packed sequences are cut into chunks and a chunk's tokens walked: plain
// arithmetic, which also compiles for the host.
//
// Token indexes are unsigned: tokens number below 2^31, and what is added to an
// index before it is compared (a step of up to 1024 tokens, a pad for each of
// up to 1024 sequences) stays below 2^32, where a signed one would wrap.
#pragma once

#ifdef __CUDACC__
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif

namespace moe {

// The sequences' tokens cut into equal chunks, where a sequence counts for `pad`
// tokens more than it has: a chunk pays for each piece it holds (its counts, its
// sums, its ticket), and with chunks of equal tokens the one with the most pieces
// sets the time (65519 x 128: 37 sequences 29.5 us, 150 36.6; with the pad 23.3
// and 28.0; 8192 x 128 in 64 sequences 24.9 and 16.3).  Sequence s takes places
// [start(s), start(s + 1)), the first pad of them without a token.
// off[0..num_seq]: the sequences' first tokens and the last one's end, rising;
// nb[0..num_seq]: sequences with tokens before each.
struct Cut {
  const int *off, *nb;
  int num_seq;
  unsigned pad, chunk;
  MOE_HD Cut(const int* off, const int* nb, int num_seq, unsigned chunks, unsigned pad)
      : off(off), nb(nb), num_seq(num_seq), pad(nb[num_seq] > 1 ? pad : 0) {
    const unsigned c = (start(num_seq) + chunks - 1) / chunks;
    chunk = c > 0 ? c : 1;
  }
  MOE_HD unsigned start(int s) const { return (unsigned)(off[s] - off[0]) + pad * (unsigned)nb[s]; }
  // the chunks that hold tokens of s (which has some)
  MOE_HD int first(int s) const { return (int)((start(s) + pad) / chunk); }
  MOE_HD int last(int s) const { return (int)((start(s + 1) - 1) / chunk); }
  // f(seq, first token, end) for every piece of chunk c
  template <class F>
  MOE_HD void pieces(unsigned c, F&& f) const {
    const unsigned all = start(num_seq), v0 = c * chunk, v1 = all < v0 + chunk ? all : v0 + chunk;
    if (v0 >= all) return;
    int lo = 0, hi = num_seq - 1;  // last s with start(s) <= v0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (start(mid) <= v0) lo = mid; else hi = mid - 1;
    }
    for (int s = lo; s < num_seq && start(s) < v1; ++s) {
      const unsigned v = start(s) + pad;  // its first token's place
      const unsigned at = (unsigned)off[s], end = (unsigned)off[s + 1];
      const unsigned a = at + (v0 > v ? v0 - v : 0), b = at + (v1 > v ? v1 - v : 0);
      if (a < b && a < end) f(s, a, b < end ? b : end);
    }
  }
};

// A lane's tokens of a piece that ends at b: t, t + step, ... below b.
struct TokenWalk {
  unsigned t, b, step;
  MOE_HD bool more() const { return t < b; }
  MOE_HD void next() { t += step; }
};

}  // namespace moe
