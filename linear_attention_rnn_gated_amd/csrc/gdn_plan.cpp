// Host-side validation and workspace layout (pure C++).
#include "gdn_plan.h"

#include <cmath>
#include <limits>

namespace gdn {

int check_shape(const gdn_shape_t* s) {
  if (!s) return GDN_ERR_INVALID_ARG;
  if (s->H_qk <= 0 || s->H_v <= 0 || s->d_k <= 0 || s->d_v <= 0 || s->C <= 0)
    return GDN_ERR_INVALID_ARG;
  if (s->qk_l2norm != 0 && s->qk_l2norm != 1) return GDN_ERR_INVALID_ARG;
  if (!std::isfinite(s->scale)) return GDN_ERR_INVALID_ARG;
  if (s->in_dtype != GDN_F32 && s->in_dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (s->H_v % s->H_qk != 0) return GDN_ERR_UNSUPPORTED;
  if (s->H_v / s->H_qk > 8) return GDN_ERR_UNSUPPORTED;  // token-step block: <= 16 waves
  if (s->d_k != s->d_v) return GDN_ERR_UNSUPPORTED;
  // keep every [.., H, d] row offset well inside 32 bits per token
  if (static_cast<int64_t>(s->H_v) * s->d_v > (1 << 20)) return GDN_ERR_UNSUPPORTED;
  for (const Claim& c : kClaims)
    if (c.d == s->d_k && c.C == s->C) return GDN_OK;
  return GDN_ERR_UNSUPPORTED;
}

int count_chunks(const int32_t* cu, int32_t n_seqs, int32_t C, Counts* out) {
  if (!cu || !out || n_seqs < 0 || C <= 0) return GDN_ERR_INVALID_ARG;
  if (cu[0] != 0) return GDN_ERR_INVALID_ARG;
  Counts r;
  for (int32_t n = 0; n < n_seqs; ++n) {
    const int64_t L = static_cast<int64_t>(cu[n + 1]) - cu[n];
    if (L < 0) return GDN_ERR_INVALID_ARG;
    r.chunks += (L + C - 1) / C;
    r.full += L / C;
  }
  r.T = cu[n_seqs];
  *out = r;
  return GDN_OK;
}

static size_t take(size_t* cursor, size_t bytes) {
  const size_t at = *cursor;
  *cursor += (bytes + kAlign - 1) / kAlign * kAlign;
  return at;
}

Layout layout(const gdn_shape_t* s, int32_t N, int64_t T, int op) {
  Layout L;
  if (check_shape(s) != GDN_OK || N < 0 || T < 0) return L;
  const size_t d = static_cast<size_t>(s->d_k), C = static_cast<size_t>(s->C);
  const size_t Hq = static_cast<size_t>(s->H_qk), Hv = static_cast<size_t>(s->H_v);
  const size_t f = sizeof(float);
  size_t cur = kAlign;  // offset 0 is never handed out
  if (op == GDN_OP_DECODE) {
    L.full_slots = N;
    L.state_slots = 0;
    L.W = take(&cur, N * Hv * C * d * f);
    L.U = take(&cur, N * Hv * C * d * f);
    L.G = take(&cur, N * Hv * C * f);
    L.total = cur;
    return L;
  }
  if (op != GDN_OP_PREFILL && op != GDN_OP_FWD_BWD && op != GDN_OP_PREFILL_CHUNKED &&
      op != GDN_OP_PREFILL_CONTINUE)
    return Layout{};
  // the continuation re-runs each sequence's up to C - 1 buffered tokens
  if (op == GDN_OP_PREFILL_CONTINUE) T += static_cast<int64_t>(N) * (static_cast<int64_t>(C) - 1);
  const bool all_chunks = op != GDN_OP_PREFILL && op != GDN_OP_PREFILL_CONTINUE;
  L.full_slots = T / static_cast<int64_t>(C);
  L.state_slots = T / static_cast<int64_t>(C) + N;
  L.cu_chunks = take(&cur, (N + 1) * sizeof(int32_t));
  L.cu_full = take(&cur, (N + 1) * sizeof(int32_t));
  // two spare token rows: the token step reads (prefetches) up to two tokens
  // past the end of a chunk; those values are never used
  L.qk = take(&cur, (T * Hq + 2) * 2 * d * f);
  const int64_t wu_slots = all_chunks ? L.state_slots : L.full_slots;
  L.W = take(&cur, wu_slots * Hv * C * d * f);
  L.U = take(&cur, wu_slots * Hv * C * d * f);
  L.G = take(&cur, wu_slots * Hv * C * f);
  L.states = take(&cur, L.state_slots * Hv * d * d * f);
  L.order = take(&cur, static_cast<size_t>(N) * sizeof(int32_t) + 1);
  if (op != GDN_OP_PREFILL_CHUNKED) L.gb = take(&cur, T * Hv * 2 * f);  // read by the token step
  if (op == GDN_OP_PREFILL_CHUNKED) L.Dl = take(&cur, L.state_slots * Hv * C * d * f);
  if (op == GDN_OP_FWD_BWD) {
    const size_t cd = L.state_slots * Hv * C * d * f;
    L.Dl = take(&cur, cd);
    L.E = take(&cur, cd);
    L.dstates = take(&cur, L.state_slots * Hv * d * d * f);
    L.dD = take(&cur, cd);
    if (d != 128) {  // at d = 128 the backward chunk kernel forms these itself
      L.SdO = take(&cur, cd);
      L.DsD = take(&cur, cd);
      L.SdD = take(&cur, cd);
    }
    L.dqv = take(&cur, T * Hv * d * f);
    L.dkv = take(&cur, T * Hv * d * f);
  }
  if (op == GDN_OP_PREFILL_CONTINUE) {
    const size_t in = s->in_dtype == GDN_BF16 ? 2 : 4;
    L.cu_ext = take(&cur, (N + 1) * sizeof(int32_t));
    L.v_ext = take(&cur, T * Hv * d * in);
    L.b_ext = take(&cur, T * Hv * f);
    L.g_ext = take(&cur, T * Hv * f);
    L.o_ext = take(&cur, T * Hv * d * f);
  }
  L.total = cur;
  return L;
}

int check_cache(const gdn_cache_t* c) {
  if (!c || !c->S_run || !c->S_chunk || !c->kbuf || !c->vbuf || !c->bbuf || !c->gbuf ||
      !c->pos)
    return GDN_ERR_INVALID_ARG;
  if (!aligned16({c->S_run, c->S_chunk, c->kbuf, c->vbuf, c->bbuf, c->gbuf, c->pos}))
    return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

bool aligned16(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0) return false;  // NULL passes
  return true;
}

int check_lru_shape(const gdn_lru_shape_t* s) {
  if (!s || s->D <= 0) return GDN_ERR_INVALID_ARG;
  if (s->gate != GDN_LRU_GATE_NONE && s->gate != GDN_LRU_GATE_COMPLEMENT && s->gate != GDN_LRU_GATE_NORM)
    return GDN_ERR_INVALID_ARG;
  if (s->in_dtype != GDN_F32 && s->in_dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (s->g_dtype != GDN_F32 && s->g_dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (s->D > (1 << 20)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

int check_lru_cache(const gdn_lru_cache_t* c) {
  if (!c || !c->S || !c->A || !c->B || !c->pos) return GDN_ERR_INVALID_ARG;
  return aligned16({c->S, c->A, c->B, c->pos}) ? GDN_OK : GDN_ERR_INVALID_ARG;
}

int64_t row_stride(int64_t ld, int64_t row) {
  if (ld == 0) return row;
  // rows past 2^40 elements apart would take offsets past 63 bits
  return ld >= row && ld <= (int64_t{1} << 40) ? ld : -1;
}

// The one pass's tile, threads and units.
//
// A block goes over its unit in rounds of threads / tile chunks, one block of
// 1024 threads a CU, so a pass takes the larger of the longest unit's rounds
// and the rounds of all units and tiles over 256 CUs, times a round's time.
// That one is longer with narrow tiles, whose rows are 16- or 32-byte pieces of
// a cache line, so that L2's request rate bounds them; measured (bf16 x, fp32 g,
// norm gate) at tiles of 8, 16, 32 and 64 channels: 33, 20, 16 and 13.5 us a round
// with all CUs at work, 27, 16.5, 12 and 10.5 with a part of them.  The tile with
// the least time is taken.
//
// Short sequences share units of up to a round: up to kLruPack sequences first
// fit, longest first, and the longest units begin first (19 sequences of 1 to 1508
// tokens x 3447 channels: 31 us, unpacked 75; 32 of 128 to 8192 x 2048: 433 us,
// unpacked 504); of more sequences, as many neighbours as fill a round on average
// (1000 of 20 tokens x 1024 channels: 66 us, a unit each 132; 2000 of 3 x 512: 30
// against 83).
//
// Blocks of 512 threads, two a CU, where all tiles and units keep them busy: one
// block's loads then overlap the other's chain (16 x 2048 tokens x 2048 channels:
// 119 us against 125; 80 x 3000 x 256: 122 against 140; with half as many blocks
// 122 against 108 us).  Smaller blocks where the batch is so small that fewer than
// 256 would be left.
static constexpr int kTile[4] = {64, 32, 16, 8};
static constexpr double kRound[4] = {13.5, 16.0, 20.0, 33.0}, kAlone[4] = {10.5, 12.0, 16.5, 27.0};
static void lru_tile(const int32_t* cu, int32_t N, int64_t chunks, int32_t D, int64_t longest, LruPlan* plan,
                     double* us) {
  *us = 0;
  for (int k = 0; k < 4; ++k) {
    const int l = kTile[k];
    const int64_t slots = kLruThreads / l;
    double rounds = 0;
    if (N <= kLruPack) {
      int64_t shorts = 0;
      for (int32_t n = 0; n < N; ++n) {
        const int64_t c = (static_cast<int64_t>(cu[n + 1]) - cu[n] + GDN_LRU_CHUNK - 1) / GDN_LRU_CHUNK;
        if (c >= slots)
          rounds += static_cast<double>((c + slots - 1) / slots);
        else
          shorts += c;
      }
      rounds += static_cast<double>((shorts + slots - 1) / slots);
    } else {
      const int64_t mean = (chunks + N - 1) / N;
      rounds = mean < slots ? static_cast<double>(chunks) / slots
                            : static_cast<double>(N) * static_cast<double>((mean + slots - 1) / slots);
    }
    const double share = rounds * ((D + l - 1) / l) / 256.0;
    const double all = (share > 1.0 ? std::ceil(share) : share) * kRound[k];
    const double one =
        static_cast<double>(((longest + GDN_LRU_CHUNK - 1) / GDN_LRU_CHUNK + slots - 1) / slots) * kAlone[k];
    const double t = all > one ? all : one;
    if (k == 0 || t < *us) {
      *us = t;
      plan->lps = l;
    }
  }
  const int64_t tiles64 = (D + 63) / 64;
  const int64_t most = longest > 0 && chunks * GDN_LRU_CHUNK * tiles64 / longest > 256 ? 512 : kLruThreads;
  const int64_t one = (longest / GDN_LRU_CHUNK + 2) * plan->lps;                    // the longest in one round
  const int64_t share = chunks * ((D + plan->lps - 1) / plan->lps) * plan->lps / 256;  // 256 blocks of the batch
  const int64_t t = ((one > share ? one : share) + 63) / 64 * 64;
  plan->threads = static_cast<int32_t>(t < most ? t : most);
}

// More than kLruPack sequences: as many neighbours a unit as fit a round with
// `each` chunks each.
static void lru_neighbours(int32_t N, int64_t each, LruPlan* plan) {
  const int64_t slots = plan->threads / plan->lps, per = each > 0 ? slots / each : kLruPack;
  plan->per = static_cast<int32_t>(per < 1 ? 1 : per > kLruPack ? kLruPack : per);
  plan->units = static_cast<int32_t>((int64_t{N} + plan->per - 1) / plan->per);
}

// Rounds of all those units and of the longest of them.
static void lru_rounds(const int32_t* cu, int32_t N, bool resume, const LruPlan& plan, int64_t* all, int64_t* worst) {
  const int64_t slots = plan.threads / plan.lps, lead = (resume ? 2 : 1) * GDN_LRU_CHUNK - 1;
  *all = *worst = 0;
  for (int64_t n0 = 0; n0 < N; n0 += plan.per) {
    const int64_t n1 = n0 + plan.per < N ? n0 + plan.per : N;
    int64_t held = 0;
    for (int64_t n = n0; n < n1; ++n) {
      const int64_t len = int64_t{cu[n + 1]} - cu[n];
      held += len > 0 ? (len + lead) / GDN_LRU_CHUNK : 0;
    }
    const int64_t r = (held + slots - 1) / slots;
    *all += r;
    *worst = r > *worst ? r : *worst;
  }
}

// Neighbours that are not alike can give a unit several long sequences one after
// another, which lru_tile's cost does not know.  Where that takes a unit more than
// twice the rounds of the longest sequence alone, the units' own time counts, with
// as many neighbours as take the least of it, the number halved for as long as that
// helps (us, without this / with it: 5000 x 1 and 10 x 8000 tokens x 512 channels
// 1196 / 532, 200 x 20 and 8 x 2000 x 256 108 / 32, both now in three steps; at up to
// twice the rounds the costs are too close: 649 of up to 298 x 2403 293 / 321).
static void lru_uneven(const int32_t* cu, int32_t N, bool resume, int32_t D, int64_t longest, LruPlan* plan, double* us) {
  int k = 0;
  while (kTile[k] != plan->lps) ++k;
  const int64_t slots = plan->threads / plan->lps;
  const int64_t alone = ((longest + (resume ? 2 : 1) * GDN_LRU_CHUNK - 1) / GDN_LRU_CHUNK + slots - 1) / slots;
  const double blocks = 256.0 * kLruThreads / plan->threads;  // at once
  double best = 0;
  for (int32_t per = plan->per; per >= 1; per /= 2) {
    LruPlan p = *plan;
    p.per = per;
    p.units = static_cast<int32_t>((int64_t{N} + per - 1) / per);
    int64_t all, worst;
    lru_rounds(cu, N, resume, p, &all, &worst);
    if (best == 0 && worst <= 2 * (alone > 1 ? alone : 1)) return;
    const double share = std::ceil(static_cast<double>(all) * ((D + p.lps - 1) / p.lps) / blocks) * kRound[k];
    const double one = static_cast<double>(worst) * kAlone[k], t = share > one ? share : one;
    if (best > 0 && t >= best) break;
    best = t;
    *plan = p;
  }
  *us = best > *us ? best : *us;
}

// Units of up to kLruPack sequences for the plan's tile and threads.
static void lru_pack(const int32_t* cu, int32_t N, bool resume, LruPlan* plan) {
  const int64_t slots = plan->threads / plan->lps;
  plan->per = 0;
  int order[kLruPack], unit[kLruPack], units = 0;
  int64_t len[kLruPack], sum[kLruPack];
  for (int n = 0; n < N; ++n) {
    len[n] = static_cast<int64_t>(cu[n + 1]) - cu[n];
    int at = n;
    for (; at > 0 && len[order[at - 1]] < len[n]; --at) order[at] = order[at - 1];
    order[at] = n;
  }
  int size[kLruPack] = {};  // sequences of each unit
  for (int i = 0; i < N; ++i) {
    // chunks, one more for the places before a resumed sequence's first token
    const int64_t need = (len[order[i]] + (resume ? 2 : 1) * GDN_LRU_CHUNK - 1) / GDN_LRU_CHUNK;
    int u = 0;
    while (u < units && sum[u] + need > slots) ++u;
    if (u == units) sum[units++] = 0;
    sum[u] += need;
    ++size[u];
    unit[i] = u;
  }
  int at = 0, next[kLruPack];
  for (int u = 0; u < units; ++u) {
    plan->first[u] = static_cast<uint8_t>(at);
    next[u] = at;
    at += size[u];
  }
  plan->first[units] = static_cast<uint8_t>(at);
  for (int i = 0; i < N; ++i) plan->seq[next[unit[i]]++] = static_cast<uint8_t>(order[i]);
  plan->units = units;
}

// The three steps read the inputs twice, 3 us per million elements, and take
// some 8 us for two launches and the chain (us, one pass / three steps: 512
// channels x 8192 tokens 42 / 30, 1024 x 4096 24 / 25, 1024 x 16384 110 / 70, 2048
// x 4096 27 / 34, 2048 x 16384 132 / 111, 4096 x 16384 163 / 201).
//
// Those costs are bf16 x's and fp32 g's with the norm gate, and stand for every
// type and gate.  fp32 x takes both ways longer alike (1024 x 16384 143 / 80, 2048 x
// 4096 33 / 38, 4096 x 16384 226 / 270; the shorter is taken in all of 12 batches);
// without a gate both are as with one.  With bf16 g the second reading costs less
// than the rule takes it for: at most 9% are lost (4096 x 16384 166 / 152, 4096 x
// 32768 319 / 289, in one pass).
bool lru_plan(const int32_t* cu, int32_t N, int64_t chunks, int32_t D, int64_t longest, bool resume, LruPlan* plan) {
  const int64_t T = N > 0 ? cu[N] : 0;
  double us;
  lru_tile(cu, N, chunks, D, longest, plan, &us);
  // over the chunks' places and whole waves, which is what the steps run over
  const double twice = 8.0 + 3e-6 * static_cast<double>(chunks * GDN_LRU_CHUNK) * ((D + 63) / 64 * 64);
  if (N > kLruPack) {
    // on average, and a resumed sequence may take a chunk more than its tokens do
    lru_neighbours(N, (chunks + N - 1) / N + (resume ? 1 : 0), plan);
    lru_uneven(cu, N, resume, D, longest, plan, &us);
  }
  if (T > GDN_LRU_SMALL && twice < us) return true;
  if (N <= kLruPack) lru_pack(cu, N, resume, plan);
  return false;
}

// The chain's rounds: 128 chunks x 32 channels in 32 KB of LDS, five blocks a CU,
// or, for longer sequences in no more blocks than CUs, where each round's latency
// is what counts, 512 chunks x 16 channels (whole prefills, us: 12 sequences to
// 14162 tokens x 200 channels 41 against 45, 16 to 14617 x 109 33 against 38; but 15
// to 4475 x 972 in 915 blocks 58 against 52), or, for many sequences of up to 64
// chunks, where blocks are what counts, 8 x 256 (whole training calls: one of 1000
// tokens and 1000 of 30, 1024 channels 206 against 368; 2000 and 100 x 100, 2048
// channels, 6464 blocks of 32 143 against 167; 2000 and 30 x 100 in 1984 blocks 69
// against 69; 41 of 2000 x 512 in 656 blocks 216 against 214).  The last also where
// blocks of 32 channels would take a launch past its threads.
int lru_chain_width(int32_t N, int32_t D, int64_t longest, int directions) {
  if (longest > 128 * GDN_LRU_CHUNK && lru_chain_blocks(N, D, 16) <= 256) return 16;
  auto fits = [&](int w) { return lru_chain_blocks(N, D, w) * directions * 256 < kLaunchThreads; };
  const bool many = longest <= 64 * GDN_LRU_CHUNK && lru_chain_blocks(N, D, 32) > 2048;
  if (!many && fits(32)) return 32;
  return fits(256) ? 256 : 0;
}

// The trainer's one pass where the longest sequence fits a round of 512 threads:
// up to 256 tokens with 64 lanes a chunk (64 x 256 tokens x 4096 channels, bf16, fp32
// g: 254 us, three steps 310; 400 x 40 x 1024: 71 against 116), to 512 with 32 (16 x
// 512 x 4096 144 against 177) and to 1024 with 16, where rows are narrow, in batches
// of up to 2^24 elements (8 x 1024 x 2048 86 against 93; 32 x 1024 x 4096 698 against
// 617).  Wider tiles are faster than narrower ones throughout, and narrower ones
// still, 8 lanes, lose to the three steps (4 x 2048 x 1024: 50 against 48).
// All with bf16 x and fp32 g.  In fp32 one pass gains more (16 x 512 x 4096 184
// against 244), with bf16 g less: 8 x 1024 x 2048, 88 against 74, loses by it.
// Batches of more than kLruPack sequences fill rounds for the longest one: those
// that would leave two thirds of the places empty take the three steps (500 tokens
// and 100 x 50, 2048 channels, seven eighths empty: 266 against 111; 250 and 300 x
// 100, 1024 channels, half empty: 175 against 233).
bool lru_train_plan(const int32_t* cu, int32_t N, int64_t chunks, int32_t D, int64_t longest, LruPlan* plan) {
  int64_t each = (longest + GDN_LRU_CHUNK - 1) / GDN_LRU_CHUNK;
  each = each > 0 ? each : 1;
  if (each > kLruTrain / 16) return false;
  plan->lps = each <= kLruTrain / 64 ? 64 : each <= kLruTrain / 32 ? 32 : 16;
  if (plan->lps == 16 && chunks * GDN_LRU_CHUNK * D > 1 << 24) return false;
  plan->threads = static_cast<int32_t>((each * plan->lps + 63) / 64 * 64);
  if (N > kLruPack)
    lru_neighbours(N, each, plan);
  else
    lru_pack(cu, N, false, plan);
  const int64_t slots = plan->threads / plan->lps;
  return plan->per == 0 || plan->units * slots <= 3 * chunks + slots;
}

int check_qk_shape(const gdn_qk_shape_t* s) {
  if (!s || s->H_q <= 0 || s->H_k < 0 || s->d <= 0 || s->r < 0 || s->r > s->d) return GDN_ERR_INVALID_ARG;
  if (s->norm != GDN_NORM_NONE && s->norm != GDN_NORM_L2 && s->norm != GDN_NORM_RMS) return GDN_ERR_INVALID_ARG;
  if (s->layout != GDN_ROPE_HALF && s->layout != GDN_ROPE_INTERLEAVED) return GDN_ERR_INVALID_ARG;
  if (!std::isfinite(s->eps) || s->eps < 0 || !std::isfinite(s->scale) || !std::isfinite(s->rope_scale) ||
      !std::isfinite(s->weight_offset))
    return GDN_ERR_INVALID_ARG;
  if (s->in_dtype != GDN_F32 && s->in_dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (s->out_dtype != GDN_F32 && s->out_dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (s->d % 8 != 0 || s->d > 512 || s->r % 8 != 0) return GDN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(s->H_q) + s->H_k > 4096) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

int64_t qk_bwd_blocks(const gdn_qk_shape_t* s, int64_t T) {
  (void)s;
  const int64_t b = (T + 3) / 4;  // a wave takes one token at a time, a block has four
  // as many as are resident at once, so that each block writes its sums once
  // (trainer 8x4096, 32 heads: 165 us; 768 blocks 170, 2048 169, 512 213)
  return b < 1024 ? b : 1024;
}

}  // namespace gdn
