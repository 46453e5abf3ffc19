// kv_attention.cu -- softmax attention over the paged NVFP4 key/value cache,
// streaming form (sm_103a): 8 or 16 (query, head) columns share one pass over
// their KV head's tokens.  One or a few queries per sequence: bound by the
// cache's bytes, with 16 columns by the latency of the few warps that their
// accumulators leave registers for.
//
// Mathematics.  For a column's query q and its visible tokens t
//   s_t = scale * q . k_t,  m = max s_t - 7 ln 2,  p_t = exp(s_t - m),
//   out = sum p_t v_t / sum p_t,  lse = m + log sum p_t,
// in one pass: a running m, l = sum p and O = sum p v, rescaled when m moves;
// partial (m, l, O) triples of disjoint token sets join by the same rescaling.
// m is only moved when a weight passes 2^15 (a score the largest one so far by 8,
// base 2), so that most tiles skip the rescaling.  The one rounding below 32 bits: the
// second product's operands are fp16, the errors 2^-11 of each weight and 2^-25 below
// the normal range, which is 2^-32 of the largest weight (m 7 above that: 2^-25, and
// 131072 tokens beside a dominant one could lose 2^-8 of the result).
//
// Both products run transposed, S^T = K Q^T and O^T = V^T P^T: the tokens
// (resp. channels) are the 16 rows of the matrix instruction and the columns
// its 8 columns, so that 8 heads sharing a KV head fill it.  The cache's codes
// become the A operand in registers: a 4-bit pair converts to half2 in one
// instruction and takes its block scale in one multiply (code * scale has 6
// significant bits and lies in [2^-10, 2688]: exact in fp16).  The contraction
// may run over the channels (tokens) in any order as long as both operands
// agree, so each lane takes the 16 bytes it loads as they are.
//
// Work: the tiles (16 tokens for each of MW groups of each of NW warps) of all
// (sequence, column group, KV head) keys, laid end to end, are cut into equal
// chunks, one per resident team; a key cut by a chunk border leaves partials in
// the workspace, joined in chunk order by csrc/kv_join.cu, so that results do not
// depend on timing.  One producer warp feeds a ring of tiles with bulk copies, a
// page of one KV head each.
//
// Measured (D = 128, 8 KV heads of 8 heads): 128 sequences of up to 8192 tokens 114
// us, 4.8 TB/s, 0.71 of the copy bandwidth (0.88 of it between the first tiles and the
// first teams to finish; the teams' times spread by 12 %, memory is not shared out
// evenly); one sequence of 131072 tokens 41 us, 3.7 TB/s; 32 sequences of up to 4096
// tokens with four queries 61 us.  A tile of 128 tokens takes a team 1.4 us with
// eight columns (three teams an SM, issue slots 60 % busy) and with sixteen (two teams:
// issue slots 44 %, matrix pipe 27 %; tiles of 64 tokens, with two teams or with three
// at 128 registers, were slower: 67.7 and 71.4 us where this took 59.5).
#include "kv_attention.cuh"
#include "../../include/nvfp4_kv_cache.h"

namespace nvr {

namespace {

// More columns of a sequence go to the tensor-memory kernel: from there on it is
// faster although it works on 128 rows whatever their number.  32 sequences of up to
// 4096 tokens, this kernel / that one, us, by columns: D = 128: 16: 38.6 / 65.1, 24:
// 64.5 / 69.7, 32: 61.1 / 65.2, 48: 83.5 / 67.1, 64: 117 / 68.4; D = 64: 24: 47.5 /
// 54.2, 32: 47.0 / 49.7, 48: 62.1 / 50.2.  Four sequences of 600: 32: 13.1 / 15.4, 64:
// 14.7 / 15.9.
constexpr int kStreamCols = 32;
// But a call of at most this many tiles an SM (128 tokens and 16 columns each, by the
// page tables' width and the window) stays here: it starts and ends sooner.  This kernel / that one,
// us: one sequence of 2 KV heads, 128 columns, 600 tokens (80 tiles) 12.6 / 14.8; 512
// columns, 1500 tokens (768) 14.9 / 17.5; four of 8 heads, 256 columns, 130 tokens (1024)
// 17.1 / 17.0; 128 columns, 600 tokens (1280) 18.3 / 16.4; 256, 600 (2560) 25.5 / 18.7.
constexpr int kStreamTiles = 6;
// Starting and ending a key (queries, joining the warps, storing) costs a team
// about as much as this many tiles: 1.5 us beside 1.4 us for a tile with eight
// columns, 3.0 beside 1.4 with sixteen (least squares over the teams of the serving
// batch and of 32 sequences with four queries).  Counted in the chunks, so that
// teams with many short keys get fewer tiles.
template <int NT>
constexpr int kKeyCost = NT;

// A key's length in the flat order: its tiles, then kKeyCost places without work.
template <int NT>
__device__ __forceinline__ int key_cost(const Group& g) { return g.tiles ? g.tiles + kKeyCost<NT> : 0; }

// What a stage of the ring holds (everything about its key, so that nothing of
// it stays in the consumers' registers); a run's first stage brings the queries.
struct alignas(16) Meta {
  uint32_t flags;
  uint32_t live;              // bit i: tokens 16 i .. 16 i + 15 of the tile were loaded
  int tile, head;
  int kv, n_q, q0, iq0, rem0, n_cols;   // the first column is head rem0 of the group's query iq0
  float k_gsa, v_gsa;
  int slot;                   // of the run's partial results
  int lo, hi;                 // the tokens that some column sees
};
// a run's first and last tile; a tile that some column does not see whole; the
// run is all of its key; the team's last run
constexpr uint32_t kFirst = 1, kLast = 2, kEdge = 4, kWhole = 8, kDone = 16;

// Byte i is 0xFF where bit i of the low four is set, and back.
__device__ __forceinline__ uint32_t bytes_of(uint32_t bits) {
  return ((bits & 15u) * 0x00204081u & 0x01010101u) * 0xFFu;
}
__device__ __forceinline__ uint32_t bits_of(uint32_t bytes) { return (bytes & 0x01010101u) * 0x10204080u >> 28; }

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
               "{%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int D, int NT, int NW, int MW, int STAGES>
struct AttnShape {
  static constexpr int kTile = 16 * NW * MW;
  static constexpr int kCols = 8 * NT;
  static constexpr int kThreads = 32 * (NW + 1);
  static constexpr int kStageBytes = kTile * D * 9 / 8;
  static constexpr int kFrag = D / 4;                        // O registers of a lane per 8 columns
  static constexpr int kShare = kFrag / NW;                  // of them, those a warp joins
  static constexpr int kJoinBytes = NW * (NW - 1) * kShare * 32 * 4;
  static constexpr int kQBytes = NT * (D / 16) * 64 * 4;
  static constexpr int kTeamBytes = (STAGES * kStageBytes + kJoinBytes + kQBytes + 2 * NW * kCols * 4 +
                               STAGES * (static_cast<int>(sizeof(Meta)) + kCols * D * 2) + (2 * STAGES + 3) * 8 + 64 + 127) / 128 * 128;
};

// A block is `TEAMS` teams of NW consumer warps and a producer, each with its own ring
// and its own share of the work.  Eight columns: three teams in a block that fills the
// SM.  (As three blocks of five warps they fit only if their fifth warps go to different
// schedulers, and beside leftovers of an earlier kernel some did not: a share then
// began when another had ended.)  Sixteen: two blocks of one team, whose registers do
// not suffice for more addressing (draft 59.5 us, as one block 64.5).
template <int D, int NT, int NW, int MW, int STAGES, int TEAMS, int BLOCKS>
__global__ void __launch_bounds__(32 * TEAMS * (NW + 1), BLOCKS)
kv_attention_kernel(const AttnParams p) {
  using Sh = AttnShape<D, NT, NW, MW, STAGES>;
  constexpr int TILE = Sh::kTile, NC = Sh::kCols, SH = Sh::kShare;
  static_assert(D == 64 || D == 128, "the fragment loads are written for these");
  static_assert(TILE <= 256 && MW == 2 && 32 * NW >= D && Sh::kStageBytes % 128 == 0, "tile plan");
  constexpr int KS = D / 16;                                 // steps of the first product
  constexpr int MT = D / 16;                                 // channel tiles of the second
  extern __shared__ uint8_t smem_raw[];
  // (uniform in the warp, and known to be)
  const int team = TEAMS == 1 ? 0 : __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x) / Sh::kThreads, 0);
  const int tid = threadIdx.x - team * Sh::kThreads, warp = tid >> 5, lane = tid & 31;
  // shares are dealt to the SMs in turn
  const int share = team * gridDim.x + blockIdx.x, shares = TEAMS * gridDim.x;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127)) +
                  team * Sh::kTeamBytes;
  float* s_join = reinterpret_cast<float*>(smem + STAGES * Sh::kStageBytes);          // [NW][NW - 1][SH][32]
  uint32_t* s_q = reinterpret_cast<uint32_t*>(s_join + Sh::kJoinBytes / 4);                 // [NT][KS][32][2]: B fragments of Q^T
  float* s_m = reinterpret_cast<float*>(s_q + Sh::kQBytes / 4);                       // [NW][NC]
  float* s_l = s_m + NW * NC;
  uint8_t* s_raw = reinterpret_cast<uint8_t*>(s_l + NW * NC);                         // [STAGES][NC][D] bf16 queries
  Meta* s_meta = reinterpret_cast<Meta*>(s_raw + STAGES * NC * D * 2);
  uint64_t* full = reinterpret_cast<uint64_t*>(s_meta + STAGES);
  uint64_t* empty = full + STAGES;
  uint64_t* meet = empty + STAGES;                           // the consumer warps' barrier: bounded, unlike bar.sync
  uint64_t* join_free = meet + 1;                            // the join buffer has been read
  int* s_start = reinterpret_cast<int*>(meet + 2);           // item, offset inside it, whether the chunk has work
  volatile int* abort_flag = s_start + 4;

  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) { mbar_init(full + s, 1); mbar_init(empty + s, NW); }
    mbar_init(meet, NW);
    mbar_init(join_free, NW);
    *abort_flag = 0;
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");

  // ---- this block's chunk of the flat order: items in order, heads inside
  // an item, tiles inside a head; each thread sums a run of items
  const int n_items = p.B * p.groups;
  const int per = (n_items + Sh::kThreads - 1) / Sh::kThreads;
  int mine = 0;
  for (int i = tid * per; i < min((tid + 1) * per, n_items); ++i) mine += key_cost<NT>(group_of<NC, TILE>(p, i)) * p.Hkv;
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += a;
  }
  int* s_scan = reinterpret_cast<int*>(s_m);                 // NW + 1 words
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w <= NW; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  const int chunk = max((total + shares - 1) / shares, kMinChunk);
  const int f0 = min(static_cast<int64_t>(share) * chunk, static_cast<int64_t>(total));
  const int f1 = min(f0 + chunk, total);
  const int excl = before + incl - mine;
  if (f0 < f1 && excl <= f0 && f0 < excl + mine) {
    int at = excl, i = tid * per;
    Group g;
    for (;; ++i) {
      g = group_of<NC, TILE>(p, i);
      const int n = key_cost<NT>(g) * p.Hkv;
      if (f0 < at + n) break;
      at += n;
    }
    s_start[0] = i;
    s_start[1] = f0 - at;
    // the last chunk may hold nothing but the last key's places without work
    const int ti = (f0 - at) % key_cost<NT>(g);
    s_start[2] = ti < g.tiles || f1 - f0 > key_cost<NT>(g) - ti;
  }
  __syncthreads();
  if (tid == 32 * NW) p.joins[share].n_parts = 0;            // (until this team turns out to start a cut key)
  if (p.cu_q && warp < NW) clear_uncovered<D>(p, share * NW + warp, shares * NW);
  if (f0 >= f1 || !s_start[2]) return;

  if (warp == NW) {
    // -------------------------------------------------------------- producer
    int item = s_start[0], off = s_start[1], f = f0, fill = 0, st = 0;
    uint32_t parity = 1;
    const int S = 1 << p.page_shift;
    const int part = min(S, TILE);                           // tokens of one copied piece
    const int pieces = TILE / part;
    bool ok = true;
    Group next = {};
    for (bool primed = false; f < f1 && ok;) {
      const Group g = next;
      // (read ahead: its loads are not waited for here)
      next = group_of<NC, TILE>(p, min(primed ? item + 1 : item, n_items - 1));
      if (!primed) {
        primed = true;
        continue;
      }
      const int cost = key_cost<NT>(g), n_item = cost * p.Hkv;
      const int32_t* table = p.page_table + static_cast<int64_t>(g.b) * p.max_pages;
      int head = off / max(cost, 1), ti = off - head * cost;
      const int iq0 = g.c0 / p.G, rem0 = g.c0 - iq0 * p.G;
      // every column sees every token of a tile inside [sure_lo, sure_hi)
      const int sure_hi = p.causal ? g.kv - g.n_q + iq0 + 1 : g.kv;
      const int sure_lo = p.window > 0 ? g.kv - g.n_q + (g.c0 + g.n_cols - 1) / p.G + 1 - p.window : 0;
      // 32 entries of the page table in the lanes, the next 32 on their way
      int at = -1, pages = -1, pages_next = -1;
      int scaled = -1;                                       // the head whose scales are at hand
      float k_gsa = 0.0f, v_gsa = 0.0f;
      auto entries = [&](int x) { return x + lane < p.max_pages ? __ldg(table + x + lane) : -1; };
      while (off < n_item && f < f1) {
        if (ti >= g.tiles) {                                 // places without work
          const int skip = min(cost - ti, f1 - f);
          off += skip; f += skip;
          ti = 0; ++head;
          continue;
        }
        const int t0 = (g.tile0 + ti) * TILE;
        const int x = t0 >> p.page_shift;                    // the tile's first page: its pages share a group of 32
        if ((x & ~31) != at) {
          pages = at >= 0 && (x & ~31) == at + 32 ? pages_next : entries(x & ~31);
          at = x & ~31;
          pages_next = entries(at + 32);
        }
        // lane i looks after piece i of the tile (at most TILE / 16 pieces)
        const int pt = t0 + lane * part;
        const int page = __shfl_sync(0xFFFFFFFFu, pages, (x & 31) + min(lane, pieces - 1));
        const bool have = lane < pieces && pt < g.hi && pt + part > g.lo && page >= 0 && page < p.n_pages;
        if (!__all_sync(0xFFFFFFFFu, wait_bounded(empty + st, parity, abort_flag))) { ok = false; break; }
        const uint32_t got = __ballot_sync(0xFFFFFFFFu, have);
        const bool first = ti == 0 || f == f0;
        if (scaled != head) {
          k_gsa = __ldg(p.k_gsa + head);
          v_gsa = __ldg(p.v_gsa + head);
          scaled = head;
        }
        if (lane == 0) {
          Meta m = {};
          m.head = head; m.tile = g.tile0 + ti;
          const int key_f0 = f - ti, key_end = key_f0 + g.tiles;
          m.kv = g.kv; m.n_q = g.n_q; m.q0 = g.q0; m.iq0 = iq0; m.rem0 = rem0; m.n_cols = g.n_cols;
          m.k_gsa = k_gsa; m.v_gsa = v_gsa; m.lo = g.lo; m.hi = g.hi;
          // slot 0 when the key's run starts with the chunk, else 1 (it ends it)
          m.slot = 2 * share + (key_f0 > f0);
          const uint32_t each = (1u << (part / 16)) - 1;
          m.live = 0;
          for (int i = 0; i < pieces; ++i)
            if ((got >> i) & 1u) m.live |= each << (i * (part / 16));
          m.flags = (first ? kFirst : 0u) | (ti == g.tiles - 1 || f == f1 - 1 ? kLast : 0u) |
                    (key_f0 >= f0 && key_end <= f1 ? kWhole : 0u) | (key_end + kKeyCost<NT> >= f1 ? kDone : 0u);
          if (key_f0 >= f0 && key_end > f1 && first)         // this block holds the key's first part
            p.joins[share] = {(key_end - 1) / chunk - key_f0 / chunk + 1, key_f0 > f0, g.q0 + iq0, rem0, g.n_cols,
                                   head, v_gsa, 0};
          if (t0 + TILE > sure_hi || t0 < sure_lo || got != (1u << pieces) - 1u) m.flags |= kEdge;
          s_meta[st] = m;
          mbar_arrive_expect_tx(full + st, __popc(got) * part * (D * 9 / 8) + (first ? g.n_cols * D * 2 : 0));
        }
        __syncwarp();
        if (have) {
          // the four regions of the page (or of the part of it in this tile) into
          // those of the tile: every lane's place in a stage is then a constant
          uint8_t* dst = smem + st * Sh::kStageBytes;
          const uint8_t* src = p.cache + (static_cast<int64_t>(page) * p.Hkv + head) * KvPage<D>::bytes(S);
          const int o = pt & (S - 1), d = lane * part;
          bulk_load(dst + d * KvPage<D>::kCodeRow, src + o * KvPage<D>::kCodeRow, part * KvPage<D>::kCodeRow, full + st);
          bulk_load(dst + KvPage<D>::key_scales(TILE) + d * KvPage<D>::kScaleRow,
                    src + KvPage<D>::key_scales(S) + o * KvPage<D>::kScaleRow, part * KvPage<D>::kScaleRow, full + st);
          bulk_load(dst + KvPage<D>::value_codes(TILE) + d * KvPage<D>::kCodeRow,
                    src + KvPage<D>::value_codes(S) + o * KvPage<D>::kCodeRow, part * KvPage<D>::kCodeRow, full + st);
          bulk_load(dst + KvPage<D>::value_scales(TILE) + d * KvPage<D>::kScaleRow,
                    src + KvPage<D>::value_scales(S) + o * KvPage<D>::kScaleRow, part * KvPage<D>::kScaleRow, full + st);
        }
        if (first) {
          // the columns of one query are heads next to each other: lane i
          // copies those of the group's i-th query
          const int iq = iq0 + lane;
          const int from = max(g.c0, iq * p.G), to = min(g.c0 + g.n_cols, (iq + 1) * p.G);
          if (from < to)
            bulk_load(s_raw + (st * NC + from - g.c0) * D * 2,
                      p.q + (g.q0 + iq) * p.q_stride + static_cast<int64_t>(head * p.G + from - iq * p.G) * D,
                      (to - from) * D * 2, full + st);
        }
        if (++st == STAGES) { st = 0; parity ^= 1u; }
        ++fill; ++off; ++f; ++ti;
      }
      off = 0;
      ++item;
    }
    if (!ok && lane == 0) {
      report_timeout(p.status);
      *abort_flag = 1;
    }
    __syncwarp();
    if (*abort_flag) {
      // copies in flight land before the block's memory goes away
      const uint64_t drain = globaltimer_ns() + 1000000000ull;
      for (int i = max(fill - STAGES, 0); i < fill; ++i)
        while (!mbar_try_wait(full + i % STAGES, (i / STAGES) & 1))
          if (globaltimer_ns() > drain) break;
    }
    return;
  }

  // ---------------------------------------------------------------- consumers
  const int r = lane >> 2, c = lane & 3;
  // this lane's places in a stage, for the warp's first 16 tokens (the other
  // tokens and fragments are constants further): key codes, both scales, value codes
  const int codes_at = warp * MW * 16 * (D / 2) + lane * (D / 8);
  const int scales_at = warp * MW * 16 * (D / 16) + (D == 128 ? 2 * lane : lane);
  const int v_codes_at = warp * MW * 16 * (D / 2) + (D == 128 ? lane * 16 : (r >> 1) * 64 + c * 16 + (r & 1) * 4);
  const int v_scales_at = warp * MW * 16 * (D / 16) + (D == 128 ? 2 * lane : (r >> 1) * 8 + 2 * c);

  float o[NT][MT][4];
  float m_neg[NT][2], l_run[NT][2], to_log2[NT][2];         // -m: +inf until a token is seen
  uint32_t met = 0;
  auto sync_consumers = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(meet);
    const bool ok = __all_sync(0xFFFFFFFFu, wait_bounded(meet, met, abort_flag));
    met ^= 1u;
    return ok;
  };
  auto give_up = [&]() {
    if (lane == 0) {
      report_timeout(p.status);
      *abort_flag = 1;
    }
  };
  const float inv_G = 1.0f / static_cast<float>(p.G);
  auto div_G = [&](int x) { return div_small(x, inv_G); };
  // the tokens [lo, hi) that column n sees
  auto sees = [&](const Meta& meta, int n, int& lo, int& hi) {
    const int pos = meta.kv - meta.n_q + meta.iq0 + div_G(meta.rem0 + min(n, meta.n_cols - 1));
    hi = n >= meta.n_cols ? 0 : p.causal ? pos + 1 : meta.kv;
    lo = p.window > 0 ? pos + 1 - p.window : 0;
  };
  uint32_t joined = 1;
  int st = 0;
  uint32_t parity = 0;
  for (bool more = true; more;) {
    if (!__all_sync(0xFFFFFFFFu, wait_bounded(full + st, parity, abort_flag))) return give_up();
    const Meta& meta = s_meta[st];
    const uint32_t flags = meta.flags;
    if (flags & kFirst) {
      const int n_cols = meta.n_cols;
      const float k_gsa = meta.k_gsa;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        // column 8 nt + r: its query row in fp16
        const bool on = 8 * nt + r < n_cols;
        const uint8_t* src = s_raw + (st * NC + 8 * nt + r) * D * 2 + c * (D / 2);
        uint32_t w[D / 8];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 u = on ? reinterpret_cast<const uint4*>(src)[i] : make_uint4(0u, 0u, 0u, 0u);
          w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
        }
        uint32_t big = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) big = max(big, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
        big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
        big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
        float up, down;
        query_scale(big, up, down);
        down *= p.scale_log2 * k_gsa;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t b[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t u = w[2 * ks + i];
            b[i] = pack_f16(__uint_as_float(u << 16) * up, __uint_as_float(u & 0xFFFF0000u) * up);
          }
          if (warp == nt % NW)
            *reinterpret_cast<uint2*>(s_q + ((nt * KS + ks) * 32 + lane) * 2) = make_uint2(b[0], b[1]);
        }
        // columns 8 nt + 2 c, + 1: what the accumulators of this lane need
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          to_log2[nt][i] = __shfl_sync(0xFFFFFFFFu, down, (2 * c + i) * 4);
          m_neg[nt][i] = INFINITY;
          l_run[nt][i] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[nt][j][i] = 0.0f;
      }
      if (!sync_consumers()) return give_up();
    }

    const uint8_t* stage = smem + st * Sh::kStageBytes;
    const uint32_t live = (meta.live >> (warp * MW)) & ((1u << MW) - 1u);
    if (live) {
      if (flags & kEdge) {
        // The weight of a token that a column does not see is 0, its value's scale must
        // not be a NaN.  A lane looks after the eight scales of one channel block of
        // tokens tg .. tg + 7: those of tokens that no column sees (stale memory, a page
        // given back, anything) become zero, and so do NaNs, which go straight to the
        // columns that do see their token.  (32 sequences with four queries 59.5 -> 60.4 us.)
        const int t0 = meta.tile * TILE + warp * MW * 16, in = lane / (D / 16) * 8, tg = t0 + in;
        uint32_t bad = 0;                                    // tokens of the warp's with a NaN
        if (in < 32) {
          uint2* at = reinterpret_cast<uint2*>(smem + st * Sh::kStageBytes + KvPage<D>::value_scales(TILE) +
                                               KvPage<D>::value_scale(warp * MW * 16 + in, lane % (D / 16)));
          const uint32_t see = (live >> (in / 16)) & 1u ? tokens32(tg, meta.lo, meta.hi) : 0u;
          const uint2 x = *at;
          const uint32_t s0 = bytes_of(see), s1 = bytes_of(see >> 4);
          const uint32_t n0 = __vcmpeq4(x.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu) & s0;
          const uint32_t n1 = __vcmpeq4(x.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu) & s1;
          *at = make_uint2(x.x & s0 & ~n0, x.y & s1 & ~n1);
          fence_proxy_async_smem();                          // (the next copy into the stage comes after)
          if (n0 | n1) bad = (bits_of(n0) | bits_of(n1) << 4) << in;
        }
        bad = __reduce_or_sync(0xFFFFFFFFu, bad);
        if (bad) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              int lo, hi;
              sees(meta, 8 * nt + 2 * c + i, lo, hi);
              if (!(bad & tokens32(t0, lo, hi))) continue;
#pragma unroll
              for (int j = 0; j < MT; ++j) o[nt][j][i] = o[nt][j][i + 2] = NAN;
            }
        }
        __syncwarp();
      }
      // --------------------------------------- S^T = K Q^T, MW times 16 tokens
      float s[MW][NT][4], s1[MW][NT][4];                     // even and odd steps: two chains of products
      uint32_t kc[MW][2][D / 32];                            // codes of tokens r, r + 8
      uint32_t sc[MW][2];                                    // their scales as half2
#pragma unroll
      for (int u = 0; u < MW; ++u) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[u][nt][i] = s1[u][nt][i] = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int tok = 16 * u + 8 * i;                    // of the warp's, for lane row 0
          if (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(stage + codes_at + tok * 64);
            kc[u][i][0] = x.x; kc[u][i][1] = x.y; kc[u][i][D / 32 - 2] = x.z; kc[u][i][D / 32 - 1] = x.w;
            sc[u][i] = e4m3x2_to_f16(
                *reinterpret_cast<const uint16_t*>(stage + KvPage<D>::key_scales(TILE) + scales_at + tok * 8));
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(stage + codes_at + tok * 32);
            kc[u][i][0] = x.x; kc[u][i][1] = x.y;
            const uint32_t b = stage[KvPage<D>::key_scales(TILE) + scales_at + tok * 4];
            sc[u][i] = e4m3x2_to_f16(b | (b << 8));
          }
        }
      }
#pragma unroll
      for (int wd = 0; wd < D / 32; ++wd) {                  // eight channels a lane: two steps
        uint32_t a[MW][2][4];
#pragma unroll
        for (int u = 0; u < MW; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t s2 = D == 128 ? __byte_perm(sc[u][i], 0, wd < 2 ? 0x1010 : 0x3232) : sc[u][i];
            e2m1x8_to_f16(kc[u][i][wd], a[u][i][0], a[u][i][1], a[u][i][2], a[u][i][3]);
#pragma unroll
            for (int x = 0; x < 4; ++x) a[u][i][x] = h2_mul(a[u][i][x], s2);
          }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int ks = 2 * wd + h;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 b = *reinterpret_cast<const uint2*>(s_q + ((nt * KS + ks) * 32 + lane) * 2);
#pragma unroll
            for (int u = 0; u < MW; ++u)
              mma16816(h ? s1[u][nt] : s[u][nt], a[u][0][2 * h], a[u][1][2 * h], a[u][0][2 * h + 1], a[u][1][2 * h + 1], b.x, b.y);
          }
        }
      }
      // ------------------------------------------------------ running softmax
      float v[MW][NT][4];                                    // scores relative to m, base 2
      auto relative = [&]() {
#pragma unroll
        for (int u = 0; u < MW; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[u][nt][i] = fmaf(s[u][nt][i], to_log2[nt][i & 1], m_neg[nt][i & 1]);
        if (flags & kEdge) {
          // token of v[0][.][0..1]; t + 8: v[0][.][2..3]
          const int t = meta.tile * TILE + warp * MW * 16 + r;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              int lo, hi;
              sees(meta, 8 * nt + 2 * c + i, lo, hi);
#pragma unroll
              for (int u = 0; u < MW; ++u)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const int ti = t + 16 * u + 8 * k;
                  if (!((live >> u) & 1u) || ti < lo || ti >= hi) v[u][nt][i + 2 * k] = -INFINITY;
                }
            }
        }
      };
#pragma unroll
      for (int u = 0; u < MW; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[u][nt][i] += s1[u][nt][i];
      relative();
      float high = -INFINITY;
#pragma unroll
      for (int u = 0; u < MW; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) high = fmaxf(high, v[u][nt][i]);
      if (__any_sync(0xFFFFFFFFu, high > kMostWeight)) {
        // set m by the largest score so far
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = -INFINITY;
#pragma unroll
            for (int u = 0; u < MW; ++u)
#pragma unroll
              for (int k = 0; k < 2; ++k)
                // (a masked score is -inf here, any other is taken from s again)
                if (v[u][nt][i + 2 * k] > -INFINITY) top = fmaxf(top, s[u][nt][i + 2 * k] * to_log2[nt][i]);
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
            const float now = fminf(m_neg[nt][i], kLift - top);
            const float shrink = now < m_neg[nt][i] ? ex2(now - m_neg[nt][i]) : 1.0f;   // ex2(-inf) = 0
            m_neg[nt][i] = now;
            l_run[nt][i] *= shrink;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              o[nt][j][i] *= shrink;
              o[nt][j][i + 2] *= shrink;
            }
          }
        relative();
      }
      uint32_t pf[MW][NT][2];                                // B fragments of P^T
#pragma unroll
      for (int u = 0; u < MW; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] = ex2(v[u][nt][i]);
          l_run[nt][0] += e[0] + e[2];
          l_run[nt][1] += e[1] + e[3];
          pf[u][nt][0] = transpose8x8(pack_f16(e[0], e[1]));
          pf[u][nt][1] = transpose8x8(pack_f16(e[2], e[3]));
        }
      // ------------------------------------------------ O^T += V^T P^T
      // Lane (r, c) holds, for tokens 2c, 2c+1 (+ 8), the 16 channels (D = 64:
      // 8 channels) of its row r; nibbles of the two tokens are interleaved so
      // that one converted pair is two tokens of one channel.
#pragma unroll
      for (int u = 0; u < MW; ++u) {
        uint32_t sv[2];
        uint32_t lo[2][D / 64], hi[2][D / 64];               // even, odd channels; bytes: channel pairs
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int tok = 16 * u + 8 * i;
          sv[i] = e4m3x2_to_f16(
              *reinterpret_cast<const uint16_t*>(stage + KvPage<D>::value_scales(TILE) + v_scales_at + tok * (D / 16)));
          const uint8_t* vc = stage + KvPage<D>::value_codes(TILE) + v_codes_at + tok * (D / 2);
          uint32_t x[D / 64], y[D / 64];                     // token 2c, token 2c + 1
          if (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4*>(vc);
            x[0] = w.x; x[D / 64 - 1] = w.y; y[0] = w.z; y[D / 64 - 1] = w.w;
          } else {
            x[0] = *reinterpret_cast<const uint32_t*>(vc);
            y[0] = *reinterpret_cast<const uint32_t*>(vc + 8);
          }
#pragma unroll
          for (int k = 0; k < D / 64; ++k) {
            lo[i][k] = (x[k] & 0x0F0F0F0Fu) | ((y[k] << 4) & 0xF0F0F0F0u);
            hi[i][k] = ((x[k] >> 4) & 0x0F0F0F0Fu) | (y[k] & 0xF0F0F0F0u);
          }
        }
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
          uint32_t a[2][2][4];                               // [token group][row half][step]
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            e2m1x8_to_f16(lo[i][k], a[i][0][0], a[i][0][1], a[i][0][2], a[i][0][3]);
            e2m1x8_to_f16(hi[i][k], a[i][1][0], a[i][1][1], a[i][1][2], a[i][1][3]);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int x = 0; x < 4; ++x) a[i][h][x] = h2_mul(a[i][h][x], sv[i]);
          }
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816(o[nt][4 * k + x], a[0][0][x], a[0][1][x], a[1][0][x], a[1][1][x], pf[u][nt][0], pf[u][nt][1]);
        }
      }
    }
    int head = 0, q0 = 0, rem0 = 0, n_cols = 0, slot = 0;
    float v_gsa = 0.0f;
    if (flags & kLast) {
      q0 = meta.q0 + meta.iq0; head = meta.head; rem0 = meta.rem0; n_cols = meta.n_cols; v_gsa = meta.v_gsa; slot = meta.slot;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + st);
    if (++st == STAGES) { st = 0; parity ^= 1u; }
    if (!(flags & kLast)) continue;
    // ------------------------------------------------ end of a run of a key
    more = !(flags & kDone);
    // join the warps: every warp gives the others their shares of its O registers
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float l = l_run[nt][i];
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 4);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
        l_run[nt][i] = l;
      }
    const bool whole = flags & kWhole;
    float* part_m = p.partials + static_cast<size_t>(slot) * NC * (D + 2);
    float* part_l = part_m + NC;
    float* part_o = part_l + NC;                             // [NC][D]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (!__all_sync(0xFFFFFFFFu, wait_bounded(join_free, joined, abort_flag))) return give_up();
      joined ^= 1u;
      if (r == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          s_m[warp * NC + 8 * nt + 2 * c + i] = -m_neg[nt][i];
          s_l[warp * NC + 8 * nt + 2 * c + i] = l_run[nt][i];
        }
      }
      float v[SH];
#pragma unroll
      for (int d = 0; d < NW; ++d) {
        float* dst = s_join + (d * (NW - 1) + (warp < d ? warp : warp - 1)) * SH * 32 + lane;
#pragma unroll
        for (int x = 0; x < SH; ++x) {
          const int reg = d * SH + x;
          const float y = o[nt][reg / 4][reg % 4];
          if (d == warp) v[x] = y;
          else dst[x * 32] = y;
        }
      }
      if (!sync_consumers()) return give_up();
      float top[2], sum[2], w_of[NW][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int n = 8 * nt + 2 * c + i;
        top[i] = s_m[n];
        sum[i] = 0.0f;
#pragma unroll
        for (int w = 1; w < NW; ++w) top[i] = fmaxf(top[i], s_m[w * NC + n]);
        const float base = top[i] == -INFINITY ? 0.0f : top[i];
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          w_of[w][i] = ex2(s_m[w * NC + n] - base);
          sum[i] += s_l[w * NC + n] * w_of[w][i];
        }
      }
      static_assert(SH >= 4 && SH % 4 == 0, "a warp joins whole pairs of channels");
      float own[2] = {0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < NW; ++w)
        if (w == warp) { own[0] = w_of[w][0]; own[1] = w_of[w][1]; }
#pragma unroll
      for (int x = 0; x < SH; ++x) v[x] *= own[x & 1];
#pragma unroll
      for (int k = 0; k < NW - 1; ++k) {
        // slot k of this warp came from warp k, or k + 1 beyond its own place
        const float w0 = k < warp ? w_of[k][0] : w_of[k + 1][0], w1 = k < warp ? w_of[k][1] : w_of[k + 1][1];
#pragma unroll
        for (int x = 0; x < SH; ++x) v[x] += s_join[((warp * (NW - 1) + k) * SH + x) * 32 + lane] * (x & 1 ? w1 : w0);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(join_free);
      // register 4 j + 2 e + i: channel (D / 8) r + 2 j + e of column 2 c + i
      const int ch = (D / 8) * r + warp * SH / 2;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int n = 8 * nt + 2 * c + i;
        if (n >= n_cols) continue;
        if (!whole) {
#pragma unroll
          for (int x = 0; x < SH / 2; x += 2)
            *reinterpret_cast<float2*>(part_o + n * D + ch + x) = make_float2(v[2 * x + i], v[2 * x + 2 + i]);
          if (r == 0 && warp == 0) {
            part_m[n] = top[i];
            part_l[n] = sum[i];
          }
          continue;
        }
        const int dq = div_G(rem0 + n);
        const int64_t row = static_cast<int64_t>(q0 + dq) * p.Hq + head * p.G + (rem0 + n - dq * p.G);
        const float inv = out_factor(v_gsa, sum[i]);
#pragma unroll
        for (int x = 0; x < SH / 2; x += 2) {
          const __nv_bfloat162 y = __floats2bfloat162_rn(v[2 * x + i] * inv, v[2 * x + 2 + i] * inv);
          *reinterpret_cast<__nv_bfloat162*>(p.out + row * D + ch + x) = y;
        }
        if (p.lse && r == 0 && warp == 0)
          p.lse[row] = lse_of(top[i], sum[i]);
      }
    }
  }
}

size_t a256(size_t v) { return (v + 255) / 256 * 256; }

struct AttnWs {
  size_t joins, partials, total;
};
AttnWs attn_ws_layout(int D) {
  AttnWs L;
  L.joins = 256;
  L.partials = a256(L.joins + kAttnMaxShares * sizeof(KeyJoin));
  L.total = a256(L.partials + size_t(2) * kPrefillMaxCtas * kPrefillCols * (D + 2) * 4);
  return L;
}

template <int D, int NT, int NW, int MW, int STAGES, int TEAMS, int BLOCKS>
nvr_status launch_attn(AttnParams& p, int max_kv, cudaStream_t s) {
  using Sh = AttnShape<D, NT, NW, MW, STAGES>;
  auto kernel = kv_attention_kernel<D, NT, NW, MW, STAGES, TEAMS, BLOCKS>;
  constexpr int kSmem = TEAMS * Sh::kTeamBytes + 128;
  static_assert(kSmem <= 227 * 1024 && BLOCKS * (kSmem + 1024) <= 228 * 1024, "shared memory");
  static bool attr_set[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return NVR_ERR_CUDA;
  const int sms = device_sm_count();
  if (sms <= 0) return NVR_ERR_CUDA;
  if (!attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return cuda_status(e);
    attr_set[dev] = true;
  }
  p.groups = static_cast<int>((static_cast<int64_t>(p.max_q) * p.G + Sh::kCols - 1) / Sh::kCols);
  // the flat order of tiles is counted in 32 bits
  const int64_t items = static_cast<int64_t>(p.B) * p.groups;
  const int64_t most = items * p.Hkv * ((max_kv + Sh::kTile - 1) / Sh::kTile + 1 + kKeyCost<NT>);
  if (items >= (int64_t(1) << 30) || most >= (int64_t(1) << 31) - (1 << 24)) return NVR_ERR_UNSUPPORTED;
  int64_t grid = sms * BLOCKS;
  if (grid * TEAMS > kAttnMaxShares) grid = kAttnMaxShares / TEAMS;
  if (grid * TEAMS * Sh::kCols > kAttnMaxCols) grid = kAttnMaxCols / Sh::kCols / TEAMS;
  if (grid > most) grid = most;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(TEAMS * Sh::kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) return cuda_status(e);
  if (max_kv <= Sh::kTile) return NVR_OK;                    // keys of one tile are never cut
  return launch_kv_join(p, D, static_cast<int>(grid) * TEAMS, Sh::kCols, items * p.Hkv, s);
}

template <int D>
nvr_status dispatch_attn(AttnParams& p, int max_kv, cudaStream_t s) {
  // Sixteen columns at a time, two teams an SM, where eight (three teams) do not hold
  // a sequence's queries: 16 columns of 32 sequences of up to 4096 tokens 38.6 us, as
  // twice eight 46.0; 32 columns 61.1 and 81.4.  Eight columns as half of sixteen: the
  // serving batch 165 us instead of 113.5, the long sequence 51 instead of 41.
  const int64_t cols = static_cast<int64_t>(p.max_q) * p.G;
  if (cols <= 8) return launch_attn<D, 1, 4, 2, 3, 3, 1>(p, max_kv, s);
  return launch_attn<D, 2, 4, 2, 3, 1, 2>(p, max_kv, s);
}

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

}  // namespace

}  // namespace nvr

using namespace nvr;

extern "C" size_t nvfp4_kv_attention_workspace_size(int64_t T_max, int64_t B_max, int Hq, int Hkv, int D) {
  if (T_max < 0 || B_max < 0 || Hkv < 1 || Hq < 1 || Hq % Hkv || !kv_head_dim_ok(D)) return 0;
  return attn_ws_layout(D).total;
}

extern "C" nvr_status nvfp4_kv_attention(const void* q, int64_t q_stride, int64_t T, int Hq, int Hkv, int D,
                                         const uint8_t* cache, int64_t n_pages, int page_size,
                                         const int32_t* page_table, int64_t B, int64_t max_pages,
                                         const int32_t* kv_lens, const int32_t* cu_q, int max_q, const float* k_gsa,
                                         const float* v_gsa, float scale, int causal, int window, void* out,
                                         float* lse, void* workspace, size_t ws_bytes, nvr_stream_t stream) {
  if (T < 0 || B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || Hkv > 65536 || Hq / Hkv > 65536) return NVR_ERR_INVALID_ARG;
  if (n_pages < 1 || max_pages < 0 || max_q < 0 || window < 0 || (window > 0 && !causal)) return NVR_ERR_INVALID_ARG;
  if (!(scale > -INFINITY && scale < INFINITY)) return NVR_ERR_INVALID_ARG;
  if (!kv_head_dim_ok(D) || !kv_page_size_ok(page_size)) return NVR_ERR_UNSUPPORTED;
  if (!cache || !k_gsa || !v_gsa || !workspace) return NVR_ERR_INVALID_ARG;
  if (T > 0 && (!q || !out || !kv_lens || B < 1 || max_q < 1 || (max_pages > 0 && !page_table)))
    return NVR_ERR_INVALID_ARG;
  if (T > 0 && (q_stride < static_cast<int64_t>(Hq) * D || q_stride % 8)) return NVR_ERR_INVALID_ARG;
  if (T > INT32_MAX || B > INT32_MAX || max_pages > (INT32_MAX - 1024) / page_size ||
      static_cast<int64_t>(max_q) * (Hq / Hkv) > INT32_MAX - 1024)
    return NVR_ERR_UNSUPPORTED;
  if (!cu_q && T != B * max_q) return NVR_ERR_INVALID_ARG;
  if (off16(q) || off16(cache) || off16(out) || off4(page_table) || off4(kv_lens) || off4(cu_q) || off4(k_gsa) ||
      off4(v_gsa) || off4(lse) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return NVR_ERR_ALIGNMENT;
  const AttnWs L = attn_ws_layout(D);
  if (ws_bytes < L.total) return NVR_ERR_WORKSPACE;
  if (T == 0) return NVR_OK;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  AttnParams p;
  p.q = static_cast<const __nv_bfloat16*>(q); p.q_stride = q_stride; p.T = T;
  p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv;
  p.cache = cache; p.n_pages = n_pages;
  p.page_shift = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
  p.page_table = page_table; p.B = static_cast<int>(B); p.max_pages = static_cast<int>(max_pages);
  p.kv_lens = kv_lens; p.cu_q = cu_q; p.max_q = max_q;
  p.k_gsa = k_gsa; p.v_gsa = v_gsa;
  p.scale_log2 = scale * 1.44269504088896341f;
  p.causal = causal != 0; p.window = window;
  p.out = static_cast<__nv_bfloat16*>(out); p.lse = lse;
  p.status = reinterpret_cast<uint32_t*>(w + kWsStatus);
  p.joins = reinterpret_cast<KeyJoin*>(w + L.joins);
  p.partials = reinterpret_cast<float*>(w + L.partials);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int max_kv = static_cast<int>(max_pages) * page_size;
  if (window >= max_kv) p.window = 0;                        // (hides nothing, and may be near 2^31)
  const int sms = device_sm_count();
  if (sms <= 0) return NVR_ERR_CUDA;
  const int64_t cols = static_cast<int64_t>(max_q) * p.G;
  // (16 columns are at most 16 queries: they see a window and 15 tokens more)
  const int seen = p.window > 0 && p.window < max_kv - 16 ? p.window + 15 : max_kv;
  const double tiles = static_cast<double>(B) * Hkv * static_cast<double>((cols + 15) / 16) * ((seen + 127) / 128);
  if (cols > kStreamCols && tiles > kStreamTiles * sms) return launch_kv_prefill(p, D, max_kv, s);
  return D == 128 ? dispatch_attn<128>(p, max_kv, s) : dispatch_attn<64>(p, max_kv, s);
}
