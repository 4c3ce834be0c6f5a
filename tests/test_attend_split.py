"""The work split of the attention kernel, compiled for the host from its own source.

The header's functions that cut a batch into per-CTA fragments (csrc/pa_attend_tc.cuh) are compiled with g++ and run over
seeded random batches: every position tile of every segment is handed out exactly once, the pieces of a cut segment are
found again (CTAs, contributions, record slots) by the arithmetic that the joining warps use, no two live records share a
slot, and every query that sees a position belongs to a segment whose tiles hold it.
"""

import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_144_gb300", "csrc")

PRELUDE = r"""
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <random>
#include <set>
#include <tuple>
#include <vector>
using std::max; using std::min;
#define __device__
#define __host__
#define __forceinline__ inline
template <typename T> T __ldg(const T* p) { return *p; }
struct AttendParams {
  const int32_t* seq_lens; const int32_t* q_starts; const int32_t* prefix_lens; const uint64_t* tree_mask;
  int max_blocks_per_seq, block_shift, num_tokens, max_q_len, group, num_kv_heads, num_seqs, window; unsigned* err;
};
struct TcParams { AttendParams a; int paired, seg_rows; };
static unsigned bits;
inline void raise_error(unsigned*, unsigned b) { bits |= b; }
enum { PA_DEVERR_SEQ_LEN = 4, PA_DEVERR_QUERY = 64 };
constexpr int kTile = 128;
constexpr int kFragCost = FRAG_COST;
"""

MAIN = r"""
#define CHECK(x) do { if (!(x)) { printf("line %d: %s (trial %d)\n", __LINE__, #x, trial); return 1; } } while (0)
int main() {
  std::mt19937 g(7);
  auto rnd = [&](int lo, int hi) { return static_cast<int>(g() % static_cast<unsigned>(hi - lo + 1)) + lo; };
  for (int trial = 0; trial < 3000; ++trial) {
    TcParams p{};
    AttendParams& a = p.a;
    const int S = rnd(1, trial % 7 == 0 ? 300 : 12), maxT = 1 << rnd(0, 13);
    a.num_seqs = S; a.num_kv_heads = rnd(1, 5); a.group = rnd(1, 8);
    a.max_q_len = trial % 3 == 0 ? 1 : rnd(1, 700); a.block_shift = 4; a.max_blocks_per_seq = (maxT + 15) / 16;
    a.window = trial % 5 == 1 ? rnd(1, 600) : 0;
    std::vector<int32_t> T(S), st(S + 1, 0), pre(S);
    for (int s = 0; s < S; ++s) {
      T[s] = rnd(0, maxT);
      const int L = rnd(0, 9) == 0 ? 0 : rnd(0, a.max_q_len);
      st[s + 1] = st[s] + (rnd(0, 5) ? min(L, T[s]) : L);   // now and then more queries than tokens
      pre[s] = rnd(0, maxT + 10);
    }
    a.num_tokens = st[S]; a.seq_lens = T.data(); a.q_starts = st.data();
    const uint64_t word = 0;
    if (trial % 5 == 2) a.prefix_lens = pre.data();
    if (trial % 5 == 3) a.tree_mask = &word;
    const int ctas = rnd(1, 2);   // of a group
    p.paired = static_cast<long long>(a.max_q_len) * a.group > stream_rows(a.group) * ctas;
    const int rpt = p.seg_rows = stream_rows(a.group) * ctas * (p.paired ? 2 : 1);
    std::vector<int> prefix(S + 1, 0);
    std::map<std::tuple<int, int, int>, std::set<int>> todo;   // tiles of every segment
    for (int s = 0; s < S; ++s) {
      const SeqView v = seq_view(a, s, true);
      int cost = 0;
      const int nm = (v.L * a.group + rpt - 1) / rpt;
      CHECK(p.paired || nm <= 1);
      for (int m = 0; m < nm; ++m) {
        const TileRange tr = tile_range(a, v, seq_prefix(a, s, v.T), rpt, m);
        cost += seg_cost(tr.hi - tr.lo);
        for (int h = 0; h < a.num_kv_heads; ++h)
          for (int t = tr.lo; t < tr.hi; ++t) todo[{s, h, m}].insert(t);
        for (int r = m * rpt; r < min((m + 1) * rpt, v.L * a.group); ++r) {
          const RowBounds b = row_bounds(a, v, seq_prefix(a, s, v.T), r / a.group);
          CHECK(b.lo >= b.hi || (tr.lo <= b.lo / kTile && (b.hi - 1) / kTile < tr.hi));
          CHECK(b.hi <= v.T || b.lo >= b.hi);
        }
      }
      prefix[s + 1] = prefix[s] + cost * a.num_kv_heads;
    }
    CHECK(bits == 0);
    const int U = prefix[S], grid = rnd(0, 3) ? 152 : rnd(1, 20);
    const int want = (U + kFragCost) / (kFragCost + 1), nw = min(grid, max(want, 1));
    if (U == 0) { CHECK(todo.empty()); continue; }
    struct Piece { int cta, tiles, kind, idx; bool whole; Frag f; };
    std::map<std::tuple<int, int, int>, std::vector<Piece>> pieces;
    for (int c = 0; c < nw; ++c) {
      FragIter it{};
      it.u = range_start(c, U, nw); it.u1 = range_start(c + 1, U, nw); it.U = U; it.nw = nw; it.s_state = -1;
      int lo = 0, hi = S - 1;
      while (lo < hi) { const int mid = (lo + hi + 1) >> 1; if (prefix[mid] <= it.u) lo = mid; else hi = mid - 1; }
      it.s = lo;
      Frag f;
      std::set<int> cut_kinds;
      int last_whole = -1;
      while (advance_frag(it, f, prefix.data(), p)) {
        auto& left = todo[{f.s, f.kvh, f.m}];
        CHECK(f.t0 < f.t1);
        for (int t = f.t0; t < f.t1; ++t) CHECK(left.erase(t) == 1);
        const int kind = slot_kind_of(f.whole, f.idx);
        if (!f.whole) CHECK(cut_kinds.insert(kind).second);       // a cut fragment has its record to itself
        pieces[{f.s, f.kvh, f.m}].push_back({c, f.t1 - f.t0, kind, f.idx, f.whole, f});
        // alternating: whole segments with records take turns, so the record before is still intact
        if (f.whole) { CHECK(kind != last_whole); last_whole = kind; } else last_whole = -1;
      }
    }
    for (auto& x : todo) CHECK(x.second.empty());
    for (auto& x : pieces) {
      const Frag& f = x.second[0].f;
      const int c0 = cta_of(f.seg_start + kFragCost, U, nw), c1 = cta_of(f.seg_start + kFragCost + f.seg_tiles - 1, U, nw);
      CHECK(c1 - c0 + 1 == static_cast<int>(x.second.size()));
      for (int c = c0; c <= c1; ++c) {
        const Piece& q = x.second[c - c0];
        CHECK(q.cta == c);
        CHECK(tiles_in(c, U, nw, f.seg_start, f.seg_tiles) == q.tiles);
        CHECK(q.whole == (c0 == c1));
        if (!q.whole) CHECK(cut_slot_kind(c, c0, U, nw, f.seg_start) == q.kind);
      }
    }
  }
  printf("ok\n");
  return 0;
}
"""


def _between(text, start, end):
    i = text.index(start)
    return text[i:text.index(end, i)]


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_work_split(tmp_path):
    with open(os.path.join(CSRC, "pa_attend.cuh")) as f:
        common = f.read()
    with open(os.path.join(CSRC, "pa_attend_tc.cuh")) as f:
        tc = f.read()
    code = PRELUDE.replace("FRAG_COST", re.search(r"kFragCost = (\d+);", tc).group(1))
    code += _between(common, "struct SeqView", "// softcap * tanh")
    code += _between(tc, "__host__ __device__ __forceinline__ int stream_rows", "// A warp's iterator").replace("struct WarpFrag", "struct Unused")
    code += _between(tc, "__device__ __forceinline__ bool advance_frag", "// The warp's next fragment")
    code += _between(tc, "// CTA whose range holds", "template <")
    code += MAIN
    src = tmp_path / "split.cpp"
    src.write_text(code)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", str(src), "-o",
                    str(tmp_path / "split")], check=True)
    r = subprocess.run([str(tmp_path / "split")], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
