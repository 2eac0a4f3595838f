"""The balance loss's cut of packed sequences into chunks and its walk over a
chunk's tokens, compiled for the host and run up to the largest call (2^31 - 1
tokens): every token is met once, inside its sequence (no GPU)."""
import subprocess
from pathlib import Path

CSRC = Path(__file__).resolve().parents[1] / "moe_expert_layer_topk_gb300" / "csrc"

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "packed_cut.cuh"

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

static unsigned rnd_state = 1;
static unsigned rnd() { return rnd_state = rnd_state * 1664525u + 1013904223u; }

static int check(const std::vector<int>& off, unsigned chunks, unsigned pad, unsigned step, bool walk_all) {
  const int n = (int)off.size() - 1;
  std::vector<int> nb(n + 1, 0);
  for (int s = 0; s < n; ++s) nb[s + 1] = nb[s] + (off[s + 1] > off[s]);
  const moe::Cut cut(off.data(), nb.data(), n, chunks, pad);
  std::vector<unsigned> at(off.begin(), off.end());  // where the next piece of each sequence has to start
  std::vector<int> seen(n, 0);
  long long row = -1;
  for (unsigned c = 0; c < chunks; ++c) {
    int bad = 0;
    cut.pieces(c, [&](int s, unsigned a, unsigned b) {
      if (bad) return;
      if (a != at[s] || b <= a || b > (unsigned)off[s + 1]) { bad = 1; return; }
      if ((long long)c + s <= row) { bad = 2; return; }
      row = (long long)c + s;
      at[s] = b;
      ++seen[s];
      if ((int)c < cut.first(s) || (int)c > cut.last(s)) { bad = 3; return; }
      if (!walk_all && b - a > 4 * step && b != (unsigned)off[n]) return;  // else: the tail of the last piece, or all of it
      const unsigned from = walk_all || b - a <= 4 * step ? a : b - 4 * step;
      unsigned long long met = 0;
      for (unsigned lane = 0; lane < step; ++lane) {
        unsigned long long turns = 0;
        for (moe::TokenWalk w{from + lane, b, step}; w.more(); w.next()) {
          if (w.t < from || w.t >= b || ++turns > (b - from) / step + 1) { bad = 4; return; }
          ++met;
        }
      }
      if (met != b - from) bad = 5;
    });
    if (bad) { std::printf("chunk %u: fault %d\n", c, bad); return 1; }
  }
  for (int s = 0; s < n; ++s) {
    CHECK(at[s] == (unsigned)off[s + 1]);
    if (off[s + 1] > off[s]) CHECK(seen[s] == cut.last(s) - cut.first(s) + 1);
  }
  return 0;
}

int main() {
  const unsigned most = 2147483647u;
  for (unsigned T : {1u, 5u, 64u, 1000u, 65519u, most - 1024, most - 511, most})
    for (int n : {1, 2, 3, 37, 1024})
      for (unsigned chunks : {1u, 2u, 152u, 304u})
        for (unsigned step : {16u, 128u, 512u})
          for (unsigned pad : {128u, step, 4 * step}) {
            for (int kind = 0; kind < 3; ++kind) {  // even, random with empty ones, all but a few tokens in the first
              std::vector<int> off(n + 1);
              for (int s = 0; s <= n; ++s) {
                unsigned long long v = (unsigned long long)T * s / n;
                if (kind == 1) v = s == 0 ? T / 50 : (s == n ? T : rnd() % T);
                if (kind == 2) v = s == 0 ? 0 : T - (T > 3u * (n - s) ? 3u * (n - s) : 0u);
                off[s] = (int)v;
              }
              for (int s = 1; s <= n; ++s)
                for (int q = s; q > 0 && off[q] < off[q - 1]; --q) { const int h = off[q]; off[q] = off[q - 1]; off[q - 1] = h; }
              if (check(off, chunks, pad, step, T <= 65519u)) {
                std::printf("T %u, %d sequences, %u chunks, pad %u, step %u, kind %d\n", T, n, chunks, pad, step, kind);
                return 1;
              }
            }
          }
  std::puts("fine");
}
"""


def test_every_token_is_met_once_up_to_the_largest_call(tmp_path):
    src, exe = tmp_path / "cut.cpp", tmp_path / "cut"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-O2", "-std=c++17", "-fwrapv", f"-I{CSRC}", "-x", "c++", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout
