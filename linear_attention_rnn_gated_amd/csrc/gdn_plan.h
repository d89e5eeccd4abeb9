// Host-side argument validation and workspace layout.  Pure C++ (no HIP), so
// the same code is built into libgdn.so and into a sanitizer-instrumented
// host test.
#pragma once

#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "gdn.h"

namespace gdn {

constexpr float kNormEps = 1e-6f;  // inside the L2 norm: x / sqrt(sum x^2 + eps)
constexpr size_t kAlign = 256;     // every workspace region starts on 256 bytes

// Shapes the library is compiled for (the "claims"): d_k == d_v == d, chunk C.
struct Claim {
  int d, C;
};
constexpr Claim kClaims[] = {{16, 16}, {128, 64}};

// Per-call counts derived from cu_seqlens on the host.
struct Counts {
  int64_t T = 0;       // total tokens
  int64_t chunks = 0;  // sum over sequences of ceil(L / C)
  int64_t full = 0;    // sum over sequences of floor(L / C)
};

// Byte offsets of the regions of one call's workspace.  A region of size 0 is
// absent.  Slots are indexed by "chunk slot": prefix sum over sequences of
// their chunk counts (all chunks for states, full chunks for W/U/G).
struct Layout {
  size_t cu_chunks = 0;  // int32 [N+1]  prefix of ceil(L/C)
  size_t cu_full = 0;    // int32 [N+1]  prefix of floor(L/C)
  size_t qk = 0;         // f32 [H_qk, T, 2, d]  normalised k, q per token
  size_t W = 0;          // f32 [full_slots, H_v, C, d]
  size_t U = 0;          // f32 [full_slots, H_v, C, d]
  size_t G = 0;          // f32 [full_slots, H_v, C]
  size_t states = 0;     // f32 [state_slots, H_v, d, d]  chunk-start states
  size_t order = 0;      // int32 [N]  sequences longest first (chunk scan)
  size_t gb = 0;         // f32 [H_v, T, 2]  (g, beta) of each value head in token order
  // trainer forward + backward only (W, U, G then use chunk slots)
  size_t Dl = 0;         // f32 [state_slots, H_v, C, d]  Delta = U - W S^T
  size_t E = 0;          // f32 [state_slots, H_v, C, d]  P^T dO
  size_t dstates = 0;    // f32 [state_slots, H_v, d, d]  gradient at chunk ends
  size_t dD = 0;         // f32 [state_slots, H_v, C, d]  dDelta, then dX_u
  size_t SdO = 0;        // f32 [state_slots, H_v, C, d]
  size_t DsD = 0;        // f32 [state_slots, H_v, C, d]
  size_t SdD = 0;        // f32 [state_slots, H_v, C, d]  then dX_w
  size_t dqv = 0;        // f32 [T, H_v, d]  per value head dq-hat
  size_t dkv = 0;        // f32 [T, H_v, d]  per value head dk-hat
  // prefill continuation only: the extended batch (buffered + new tokens of
  // every sequence, T' <= T + N (C - 1) rows) and its outputs
  size_t cu_ext = 0;     // int32 [N+1]  prefix of buffered + new tokens
  size_t v_ext = 0;      // in_dtype [T', H_v, d]
  size_t b_ext = 0;      // f32 [T', H_v]
  size_t g_ext = 0;      // f32 [T', H_v]
  size_t o_ext = 0;      // f32 [T', H_v, d]
  size_t total = 0;
  int64_t full_slots = 0, state_slots = 0;
};

// GDN_OK, GDN_ERR_INVALID_ARG or GDN_ERR_UNSUPPORTED.
int check_shape(const gdn_shape_t* s);

// Validates cu_seqlens on the host (starts at 0, non-decreasing) and counts
// tokens and chunks.  GDN_OK or GDN_ERR_INVALID_ARG.
int count_chunks(const int32_t* cu_host, int32_t n_seqs, int32_t C, Counts* out);

// Workspace layout for an op, sized from (n_seqs, total_tokens) only, so that
// gdn_workspace_bytes needs no cu_seqlens: slots are bounded by T/C + N.
Layout layout(const gdn_shape_t* s, int32_t n_seqs, int64_t total_tokens, int op);

// Checks the pointer fields of a decode cache (all must be non-NULL).
int check_cache(const gdn_cache_t* c);
// True if every pointer is 16-byte aligned (NULL counts as aligned).
bool aligned16(std::initializer_list<const void*> ptrs);

// Gated linear recurrence.  Channels per decode-cache position counter.
constexpr int32_t kLruGroup = 256;
int check_lru_shape(const gdn_lru_shape_t* s);
// All fields of a recurrence cache non-NULL and aligned.
int check_lru_cache(const gdn_lru_cache_t* c);
// A row distance as given (0 = dense): the distance, or -1 if it is too small.
int64_t row_stride(int64_t ld, int64_t row);
// Chunk slots of T tokens in N sequences, whatever their lengths and whichever
// of them begin inside a chunk.
inline int64_t lru_slots(int64_t T, int64_t N) { return T / GDN_LRU_CHUNK + 2 * N; }

// How a prefill runs (see gdn_lru.hip).
constexpr int kLruPack = 64;       // most sequences of a unit, and those that are sorted into units
constexpr int kLruThreads = 1024;  // most threads of a one-pass block
constexpr int kLruTrain = 512;     // and of the trainer's
struct LruPlan {
  int32_t lps = 64;       // lanes per chunk = channels of a block's tile: 8, 16, 32 or 64
  int32_t threads = 64;   // of a block: a multiple of 64
  int32_t units = 0;      // groups of sequences that a block takes
  int32_t per = 0;        // 0: unit u is the sequences seq[first[u]] .. seq[first[u + 1] - 1];
                          // else it is `per` neighbours, those from u per on
  uint8_t seq[kLruPack] = {};
  uint8_t first[kLruPack + 1] = {};
};
// Fills the plan of the one pass from a validated cu_seqlens with its count of
// chunks (each sequence's from its first token) and its longest length; true
// where the three steps are expected to be faster.
bool lru_plan(const int32_t* cu_host, int32_t n_seqs, int64_t chunks, int32_t D, int64_t longest, bool resume,
              LruPlan* plan);

// A launch holds fewer threads than this.
constexpr int64_t kLaunchThreads = int64_t{1} << 32;
// Blocks of a chain of `width` channels a block, and the width to launch in one
// or two directions: 16, 32 or 256, or 0 where no launch holds it.
inline int64_t lru_chain_blocks(int64_t N, int64_t D, int width) { return N * ((D + width - 1) / width); }
int lru_chain_width(int32_t n_seqs, int32_t D, int64_t longest, int directions);

// Fills the plan of the trainer's one pass; false where the three steps are
// expected to be faster or a sequence does not fit one round.
bool lru_train_plan(const int32_t* cu_host, int32_t n_seqs, int64_t chunks, int32_t D, int64_t longest, LruPlan* plan);

// Norms of q and k with rotary positions.
int check_qk_shape(const gdn_qk_shape_t* s);
// Blocks of the gradient kernel that keep partial weight sums (a function of
// the sizes alone).
int64_t qk_bwd_blocks(const gdn_qk_shape_t* s, int64_t T);

}  // namespace gdn
