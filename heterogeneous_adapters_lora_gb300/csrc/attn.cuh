// Internal definitions of the attention calls: the plan's arrays, the
// arguments of the kernels, and what they share.
//
// A plan cuts a batch into *tiles* (up to 2 x kTileRows rows of one problem,
// a row being one query token and one of the query heads that share a
// key/value head) and each tile's keys into ranges of kBlock keys, one *item*
// per range and key/value head.  A problem is a sequence with its own keys or
// a group with its prefix.  A tile with one range and no prefix is written
// where it belongs; every other item leaves a partial result (normalised
// output and log2 of its softmax sum, fp32), and the join kernel adds the
// partial results of each token up.
#pragma once

#include "lora_internal.cuh"

namespace attn {

constexpr int kTileRows = 128;  // rows of one MMA tile; an item has up to two
constexpr int kBlock = 128;     // keys of a block
constexpr int kMostKeys = 1 << 30;  // of a sequence or prefix: block ends stay within 32 bits

constexpr int kMostRows = 0x7fffff00;  // of keys and values: boxes that begin past them end within 32 bits

// How long a unit takes a CTA, in tenths of a microsecond: a block of keys of
// an item of two row tiles (bound by the products and the softmax), a block of
// an item of one (by HBM, two such streams at a time), and what an item takes
// beside its blocks.
constexpr int kSms = 152;
constexpr int kPairBlock = 18, kPairItem = 20, kOneBlock = 16, kOneItem = 10;

// Ranges of keys: with the batch's time spread evenly over the SMs, a range of
// a two-tile item takes at most one SM's share, one of a one-tile item, whose
// partial results are small, half of it.  None has less than kMinBlocks blocks
// unless its tile has no more, a prefix's one less.  But when ranges no longer
// than kMostFit leave every CTA at most one unit, the shortest such ranges are
// taken, of kMinOwnBlocks or, for prefixes, whose results are joined in any
// case, kMinPrefixBlocks at least (a token behind a prefix of 8000: 18.3 us in
// 21 ranges of 3 blocks, 176 units, 15.7 in 16 of 4; 4 tokens behind one of 1000:
// 11.4 in ranges of 3, 10.6 of 2; 16 tokens over 4000 keys 14.3 of 4, 13.5 of 3).
// Batches of more tiles than SMs are not looked at, and tiles whose own keys the
// join takes count: without them 152 to 256 tokens of up to 16 own keys behind a
// prefix of 500 take 13.0 to 20.2 us instead of 13.9 to 20.0, but behind one of
// 1000, where there is more to join, 19.7 to 23.5 instead of 15.0 to 22.9.
constexpr int kMinBlocks = 4;
constexpr int kMostFit = 16, kMinOwnBlocks = 3, kMinPrefixBlocks = 2;

// In batches with prefixes, own keys of a sequence of one token that are no
// more than this need no item, nearly empty tiles that cost a CTA 4 us a pair:
// the join takes them as it does partial results, a dependent round of three
// keys after another (256 tokens behind a prefix of 500: up to 10 own keys 41 us
// with items, 18 without; up to 60 own keys 41 and 37; of up to 24 or 32 keys it
// is slower where few tokens have so few, 32 prefixes 111 and 113 against 108).
constexpr int kShortKeys = 16;

// One item of a plan (8 words).  The items of two row tiles come first, then
// those of one, each kind longest first.
struct Item {
    int tok0, n_tok;  // its query tokens
    int prob;         // sequence b, or -1 - g for the prefix of group g
    int blk0, blk1;   // its blocks of keys
    int kv_len;       // keys of the problem
    int lim0;         // keys that its first token sees (causal: + 1 for each token on; may be < 1)
    int part;         // token row of its partial result, -1: the result goes to the output
};
static_assert(sizeof(Item) == 32, "plan items are 8 words");

// counters[] of a plan; at kBinding (8 bytes) the binding that the status word belongs to
enum { kItems = 0, kPartTokens = 1, kTiles = 2, kStatus = 3, kUnits = 4, kJoins = 5, kBinding = 6 };

// A unit is what a CTA works on at a time, for one key/value head: an item of
// two row tiles, or one or two items of one tile.  Units come the longest
// first, and hold their items, so that one read tells all of the next one.
struct Unit {
    Item item[2];  // item[1].n_tok is 0 when there is one
};

// tokens of an item's first or second row tile, and of an item
__host__ __device__ inline int tile_tokens(int group) { return kTileRows / group; }

struct Args {
    const Unit *units;
    const int32_t *counters;
    int32_t *tickets;  // [0] units taken beyond each CTA's first, [1] CTAs done; zero between calls
    int32_t *status;
    int hq, hkv, G, D, page, causal, T;
    float scale_log2;  // scale * log2(e)
    const uint16_t *q, *k, *v;
    long long ldq, ldk, ldv, n_rows, ldo;
    const int32_t *table, *ptable;
    long long ld_table, ld_ptable;
    uint16_t *out;
    // Partial results: a slot of nt tokens has, per key/value head, nt * G rows from
    // row part * hq + head * nt * G on; its outputs lie as [D / 8][rows][8], so that
    // the warps, with a row per lane, store them in one piece and heads are read side by side.
    float *part_o;
    float *part_lse;
};

}  // namespace attn

// Launch the item kernel (attn.cu).
lora_status_t lora_attn_launch(const attn::Args &a, int max_items, cudaStream_t s);
