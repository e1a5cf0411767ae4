// How a call of the paged attention is divided over workgroups: arithmetic on its
// counts and bounds, shared by the launches and, as plain C++, by the checks on
// the host.
#pragma once

namespace gdn {

constexpr int kTileKeys = 64;           // keys a wave takes at once
constexpr int kTileRows = 16;           // rows of a workgroup of the few-rows kernel
constexpr int kManyRows = 128;          // of the many-rows kernel

// Which requests a launch takes: all, those of at most kSmallRows rows per kv
// head, or the larger ones.
enum class Take { kAll, kSmall, kLarge };
constexpr int kSmallRows = 32;

constexpr int kCUs = 256;

// What a format's kernels and their measured times decide of it: the least keys
// of a part of the few-rows kernel, of the same where three of four CUs are
// idle, and of the many-rows kernel; waves of a workgroup of both kinds of rows;
// workgroups of it that all CUs hold at once.
struct SplitRules {
    int min_chunk, idle_chunk, many_chunk;
    int waves, room, many_rows = kManyRows;
};

struct Launch {
    long long units;        // (row tile, kv head) pairs, upper bound; 0: none
    long long rows;         // of partial results
    int chunk, splits;
    long long floats;       // of partial results
};

struct Plan {
    Take few_takes;
    bool by_rows;
    Launch few, many;
};

// ---------------------------------------------------------------------------
// With at most a token per request on average the few-rows kernel takes
// everything; else it takes the requests of up to kSmallRows rows, and the
// many-rows kernel the others (16 rows of a wave cost it as much as 32, and it
// reads a key once for 128 rows).  Keys are split until there is a workgroup for
// every CU, or as many of the many-rows kernel's as fit at once, but into parts of
// the rules' least keys or more.
// ---------------------------------------------------------------------------
inline Launch divide(long long tiles, long long busy, long long rows, int kv_heads, int d, int max_seq_len, int aim,
                     long long min_chunk) {
    Launch p{tiles * kv_heads, rows, 0x40000000, 1, 0};
    busy *= kv_heads;
    long long want = busy > 0 ? aim / busy : 1;
    const long long most = max_seq_len / min_chunk;
    if (want > most) want = most;
    if (want > 1) {
        const long long chunk = ((max_seq_len + want - 1) / want + kTileKeys - 1) / kTileKeys * kTileKeys;
        p.splits = (int)((max_seq_len + chunk - 1) / chunk);
        if (p.splits > 1) {
            p.chunk = (int)chunk;
            p.floats = rows * p.splits * (d + 2);
        }
    }
    return p;
}

// window: 0, or the keys that a row sees at most (a plan needs no more workspace for it)
inline Plan plan_of(const SplitRules &rules, long long T, long long S, int q_heads, int kv_heads, int d, int max_seq_len,
                    int window = 0) {
    const long long G = q_heads / kv_heads;
    // few rows that see no more than one part's keys are not split, wherever these lie and
    // however few keys a part may have
    const int few_len = window > 0 && window <= rules.min_chunk ? 1 : max_seq_len;
    Plan p{};
    if (T <= S) {
        p.few_takes = Take::kAll;
        const long long full = T * G / kTileRows;
        const long long busy = full > T ? full : T;
        p.few = divide(full + S, busy, T * q_heads, kv_heads, d, few_len, kCUs,
                       busy * kv_heads * 4 <= kCUs ? rules.idle_chunk : rules.min_chunk);
    } else {
        p.few_takes = Take::kSmall;
        const long long full = T * G / rules.many_rows, busy = full > 1 ? full : 1, room = rules.room;
        // the small requests' parts need not be shorter than what the other
        // workgroups take anyway: at least this many keys one after the other, where
        // a small request's waves share theirs
        const long long anyway = busy * kv_heads * (T / S) / 2 / room * rules.waves;
        p.few = divide(S * (kSmallRows / kTileRows), S, S * kSmallRows * kv_heads, kv_heads, d, few_len, kCUs,
                       anyway > rules.min_chunk ? anyway : rules.min_chunk);
        // the fewer tile numbers of two ways that are enough (a request of many rows has
        // more than kSmallRows): 29 decode rows and 16 tokens take 23 us with 3 per kv
        // head, 32 with 31
        const long long by_rows = T * G / kSmallRows + 1;
        p.by_rows = by_rows < full + S;
        p.many = divide(p.by_rows ? by_rows : full + S, busy, T * q_heads, kv_heads, d, max_seq_len, room, rules.many_chunk);
    }
    return p;
}

}  // namespace gdn
