// Attention over the rows of variable-length sequences and its gradients.
#include "fpstok_mma.h"
#include "fpstok_seqs.h"

namespace fpstok {

constexpr float kLog2e = 1.44269504088896f, kLn2 = 0.693147180559945f;

// The rows of one workgroup's tile.  A row is a (query, head of the group) pair
// of one key head, numbered query * G + head: every row of a tile reads the
// same keys, so one query of 8 heads is 8 rows of a tile, and K and V are read
// once for the group.
struct RowTile {
    int64_t q0, k0;  // first buffer rows of the sequence
    int tq, tk, row0, rows;  // rows: those of the tile that exist
    int pad;                 // rows of the tile inside a padded sequence's slots
    int hk, b, part;  // part: of a split walk
};

// Decodes a workgroup's place in the grid: heads fastest, so that with 8 key
// heads (or a multiple) a head's tiles stay on one of the 8 XCDs and share its
// L2.
// KEYS: the tile is of keys (G = 1), not of rows of queries.
// Of a walk split into `parts`, the parts of one tile are neighbours (a stride
// between them would give a compute unit the same tile's again and again).
template <int SHIFT, bool KEYS>
__device__ __forceinline__ bool row_tile(const AttnArgs& a, int parts, RowTile& t) {
    const SeqArgs& s = KEYS ? a.ks : a.qs;
    const int G = KEYS ? 1 : a.G;
    const uint32_t place = blockIdx.x / (uint32_t)a.Hk;
    t.hk = (int)(blockIdx.x - place * (uint32_t)a.Hk);
    uint32_t slot = place, slots = gridDim.x / (uint32_t)a.Hk;
    t.part = 0;
    if (parts > 1) {
        slot = place / (uint32_t)parts;
        slots /= (uint32_t)parts;
        t.part = (int)(place - slot * (uint32_t)parts);
    }
    // later rows see more keys where only the right is bounded: those first
    if (!KEYS && a.right >= 0 && a.left < 0) slot = slots - 1 - slot;
    int64_t start, tile;
    int len;
    if (s.cu) {
        t.b = find_seq(s, slot, G, SHIFT, start, len, tile);
        if (tile < 0) return false;
    } else {
        const uint32_t per = (uint32_t)(((int64_t)s.cap * G + (1 << SHIFT) - 1) >> SHIFT);
        t.b = (int)(slot / per);
        tile = slot % per;
        seq_rows(s, t.b, start, len);
    }
    const int64_t left = (int64_t)len * G - (tile << SHIFT);
    if (s.cu && left <= 0) return false;
    const int64_t pad = s.cu ? 0 : (int64_t)s.cap * G - (tile << SHIFT);
    int64_t start2 = start;
    int len2 = len;
    if (!a.same_seqs) seq_rows(KEYS ? a.qs : a.ks, t.b, start2, len2);
    t.q0 = KEYS ? start2 : start;
    t.tq = KEYS ? len2 : len;
    t.k0 = KEYS ? start : start2;
    t.tk = KEYS ? len : len2;
    t.row0 = (int)(tile << SHIFT);
    t.rows = left < 0 ? 0 : left < (1 << SHIFT) ? (int)left : 1 << SHIFT;
    t.pad = pad < (1 << SHIFT) ? (int)pad : 1 << SHIFT;
    return true;
}

// Keys that some row with a place in [pa, pb] sees, in tiles of BN: `sink`
// tiles from key 0 on, then tiles first .. first + count - sink - 1.  (Rows
// stay below 2^30 and windows below the rows, so places fit in 32 bits.)
template <int BN>
struct KeyTiles {
    int sink, first, count, from = 0;
    __device__ __forceinline__ KeyTiles(const AttnArgs& a, int pa, int pb, int tk) {
        int hi = tk - 1, lo = 0;
        if (a.right >= 0 && pb + a.right < hi) hi = pb + a.right;
        if (a.left >= 0 && pa - a.left > 0) lo = pa - a.left;
        first = lo / BN;
        sink = 0;
        count = 0;
        if (hi >= 0) {
            const int last = hi / BN;
            const int n = a.sinks < hi + 1 ? a.sinks : hi + 1;
            sink = (n + BN - 1) / BN;
            if (sink > first) sink = first;
            count = sink + (last >= first ? last - first + 1 : 0);
        }
    }
    __device__ __forceinline__ int tile(int i) const {
        i += from;
        return i < sink ? i : first + i - sink;
    }
    // Keeps the tiles of part `split` of `splits` and returns their number.
    __device__ __forceinline__ int part(int split, int splits) {
        if (splits == 1) return count;
        const int per = (int)(((uint32_t)count + (uint32_t)splits - 1) / (uint32_t)splits);
        from = split * per < count ? split * per : count;
        return count - from < per ? count - from : per;
    }
};

// How the keys j0 .. j0 + BN - 1 look to rows with places in [pa, pb]: 0 no
// row sees any, 1 some rows hide some, 2 every row sees all.
template <int BN>
__device__ __forceinline__ int tile_view(const AttnArgs& a, int pa, int pb, int tk, int j0) {
    const int j1 = j0 + BN - 1;
    const bool left_all = a.left < 0 || j0 >= pb - a.left || j1 < a.sinks;
    const bool left_none = a.left >= 0 && j1 < pa - a.left && j0 >= a.sinks;
    const bool right_all = j1 < tk && (a.right < 0 || j1 <= pa + a.right);
    const bool right_none = j0 >= tk || (a.right >= 0 && j0 > pb + a.right);
    return left_none || right_none ? 0 : left_all && right_all ? 2 : 1;
}

// tile_view for many tiles of the same rows: ranges of j0.
template <int BN>
struct View {
    int pa, pb, tk, all_lo, any_lo;
    uint32_t all_span, any_span;
    __device__ __forceinline__ View(const AttnArgs& a, int pa, int pb, int tk)
        : pa(pa), pb(pb), tk(tk) {
        int hi = tk - BN;
        if (a.right >= 0 && pa + a.right - (BN - 1) < hi) hi = pa + a.right - (BN - 1);
        all_lo = a.left >= 0 && pb - a.left > 0 ? pb - a.left : 0;
        all_span = (uint32_t)(hi - all_lo);
        if (hi < all_lo) all_lo = 0x7fffffff, all_span = 0;
        hi = tk - 1;
        if (a.right >= 0 && pb + a.right < hi) hi = pb + a.right;
        any_lo = a.left >= 0 && pa - a.left - (BN - 1) > 0 ? pa - a.left - (BN - 1) : 0;
        any_span = (uint32_t)(hi - any_lo);
        if (hi < any_lo) any_lo = 0x7fffffff, any_span = 0;
    }
    __device__ __forceinline__ int of(const AttnArgs& a, int j0) const {
        if (j0 < a.sinks) return tile_view<BN>(a, pa, pb, tk, j0);
        return (uint32_t)(j0 - all_lo) <= all_span ? 2 : (uint32_t)(j0 - any_lo) <= any_span;
    }
};

// The keys one row sees: [lo, lo + span] and those below `sink`.
struct Window {
    int lo, sink;
    uint32_t span;
    __device__ __forceinline__ Window(const AttnArgs& a, int p, int tk) {
        const int hi = a.right >= 0 && p + a.right < tk - 1 ? p + a.right : tk - 1;
        lo = a.left >= 0 && p - a.left > 0 ? p - a.left : 0;
        sink = a.sinks < hi + 1 ? a.sinks : hi + 1;
        span = hi - lo;
        if (hi < lo) lo = 0x7fffffff, span = 0;  // none: no key has that number
    }
    __device__ __forceinline__ bool hides(int j) const {
        return ((uint32_t)(j - lo) > span) & (j >= sink);
    }
    // Registers of a transposed block of 32 keys from key j0 on (half: lane >> 5)
    // whose key the row does not see become `fill`.  No key at or past `sinks`
    // is a sink, so most tiles need one comparison per key.
    __device__ __forceinline__ void mask(f32x16& x, int j0, int half, int sinks, float fill) const {
        const int jb = j0 + half * 4;
        if (j0 >= sinks) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int at = (e >> 2) * 8 + (e & 3);
                x[e] = (uint32_t)(jb - lo + at) > span ? fill : x[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = hides(jb + (e >> 2) * 8 + (e & 3)) ? fill : x[e];
        }
    }
};

// The rows (keys or queries) that lost infinite or not-a-number elements in
// the tiles of a workgroup's walk: a bit for each tile, modulo 32, and for
// each row of it.  A tile whose number modulo 32 is another's may show rows of
// that one too: whoever looks tests the elements themselves.
struct BadRows {
    uint32_t tiles;
    uint32_t rows[32][2];
    __device__ __forceinline__ void clear(int tid) {
        if (tid < 64) rows[tid >> 1][tid & 1] = 0;
        if (tid == 64) tiles = 0;
    }
    __device__ __forceinline__ void note(int tile, int row) {
        atomicOr(&rows[tile & 31][row >> 5], 1u << (row & 31));
        atomicOr(&tiles, 1u << (tile & 31));
    }
    // Rows of a tile, the same in every lane.
    __device__ __forceinline__ uint64_t of(int tile) const {
        const uint32_t lo = __builtin_amdgcn_readfirstlane(rows[tile & 31][0]);
        const uint32_t hi = __builtin_amdgcn_readfirstlane(rows[tile & 31][1]);
        return (uint64_t)hi << 32 | lo;
    }
};

// The sum of the infinite and not-a-number elements of rows, or, ZERO, of 0
// times them, for the result of a row that sees them, where a tile that other
// rows do not see whole was multiplied without them.  The two halves of a wave
// take every other 16 bytes of the 64 elements from d0 on.  Rare, so it works
// on the stored result.  (Window of 256, 55k pulses, 8 heads on 4, an infinite
// element in 1 of 100 rows of grad_out: 286 us a backward pass, 240 without any; in
// every row 1.27 ms.  Element by element over all rows of such tiles: 17 and 18 ms.)
template <class T, bool ZERO = false>
struct BadSum {
    static constexpr int V = 16 / (int)sizeof(T), C = 64 / (2 * V);
    float sum[C * V];
    int d0;
    __device__ __forceinline__ BadSum(int d0) : d0(d0) {
#pragma unroll
        for (int e = 0; e < C * V; ++e) sum[e] = 0.0f;
    }
    __device__ __forceinline__ void add(const T* src, int D, int half) {
        u32x4 x[C];
        bool bad = false;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int d = d0 + (2 * c + half) * V;
            x[c] = *(const u32x4*)(src + (d < D ? d : 0));
        }
#pragma unroll
        for (int c = 0; c < C; ++c) bad |= chunk_bad<T>(x[c]);
        if (!bad) return;
        using Vec = T __attribute__((ext_vector_type(V)));
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const Vec v = __builtin_bit_cast(Vec, x[c]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float y = (float)v[e];
                const bool hit = (__float_as_uint(y) & 0x7f800000u) == 0x7f800000u;
                sum[c * V + e] += !hit ? 0.0f : ZERO ? NAN : y;
            }
        }
    }
    template <class TO>
    __device__ __forceinline__ void store(TO* dst, int D, int half) const {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int d = d0 + (2 * c + half) * V;
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (d < D && sum[c * V + e] != 0.0f)
                    dst[d + e] = (TO)((float)dst[d + e] + sum[c * V + e]);
        }
    }
};

// Row `p` of D elements as operands of STEPS product steps, zero where it is
// not `live` (its lanes load `any`, a row that exists: loads under a divergent
// branch would be waited for one by one).
template <class T, int STEPS>
__device__ __forceinline__ void load_row(typename Elem<T>::Frag* f, const T* p, bool live,
                                         const T* any, int D, int half) {
    using Frag = typename Elem<T>::Frag;
    p = live ? p : any;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int d = s * 16 + half * 8;
        f[s] = *(const Frag*)(p + (d < D ? d : 0));
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const bool has = live && s * 16 + half * 8 < D;
        u32x4* x = (u32x4*)&f[s];
#pragma unroll
        for (int e = 0; e < (int)sizeof(Frag) / 16; ++e) x[e] = has ? x[e] : 0;
    }
}

// The rows of one workgroup, its waves and its lanes (32 rows per wave across
// the lanes, both halves of a wave the same 32), and their places among the
// keys.  `first_row`: the first row of this wave's 32 in the tile.
struct QueryRows {
    int r, qi, h, pa, pb, wa, wb;
    int64_t row;
    bool live;
    __device__ __forceinline__ QueryRows(const AttnArgs& a, const RowTile& t, int first_row,
                                         int lane) {
        const int G = a.G;
        // row / G: a shift where the group is a power of two
        auto query = [&](int row) {
            return a.g_shift >= 0 ? row >> a.g_shift : (int)((uint32_t)row / (uint32_t)G);
        };
        r = first_row + (lane & 31);
        qi = query(t.row0 + r);
        h = t.hk * G + (t.row0 + r) - qi * G;
        live = r < t.rows;
        row = t.q0 + qi;
        const int off = t.tk - t.tq, last = t.rows > 0 ? t.rows - 1 : 0;
        const int wl = first_row + 31 < last ? first_row + 31 : last;
        pa = query(t.row0) + off;
        pb = query(t.row0 + last) + off;
        wa = query(t.row0 + first_row) + off;
        wb = query(t.row0 + wl) + off;
    }
    // This lane's row of a view, as operands of STEPS product steps.
    template <class T, int STEPS>
    __device__ __forceinline__ void load(typename Elem<T>::Frag* f, const HeadsArg& v, int D,
                                         int half) const {
        load_row<T, STEPS>(f, (const T*)v.data + row * v.row + h * v.head, live, (const T*)v.data,
                           D, half);
    }
};

// BadSum over the keys that a lane's row sees of the tiles that the workgroup's
// rows do not all see whole, added to `dst`.
template <int BN, bool ZERO = false, class T, class TO>
__device__ __forceinline__ void add_bad_keys(TO* dst, const AttnArgs& a, const KeyTiles<BN>& kt,
                                             int n, const BadRows& bad, const QueryRows& q, int tk,
                                             const Window& w, bool live, int half, const T* base,
                                             int64_t stride) {
#pragma unroll 1
    for (int d0 = 0; d0 < a.D; d0 += 64) {
        BadSum<T, ZERO> sum(d0);
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const int j0 = kt.tile(i) * BN;
            if (tile_view<BN>(a, q.pa, q.pb, tk, j0) != 1) continue;
#pragma unroll 1
            for (uint64_t rows = bad.of(i); rows != 0; rows &= rows - 1) {
                const int j = j0 + __builtin_ctzll(rows);
                if (live && j < tk && !w.hides(j)) sum.add(base + j * stride, a.D, half);
            }
        }
        if (live) sum.store(dst, a.D, half);
    }
}

// A result's registers become zero in lanes where `keep` is false (what they
// hold may not be finite); one test if there are none.
template <int DB>
__device__ __forceinline__ void zero_unless(f32x16* x, bool keep) {
    if (__all(keep)) return;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int e = 0; e < 16; ++e) x[db][e] = keep ? x[db][e] : 0.0f;
}

// A row's running maximum (m, and mc = m * c as subtracted), sum and result.
// The maximum a row subtracts is moved only when it grew by more than 2^8 (a
// rescale costs as many multiplications as the result has registers); weights
// stay below 2^8.
template <class T, int DB>
struct Softmax {
    float m = -INFINITY, mc = 0.0f, l = 0.0f;
    f32x16 o[DB];
    __device__ __forceinline__ Softmax() {
#pragma unroll
        for (int db = 0; db < DB; ++db) o[db] = 0.0f;
    }
    // Takes the maximum of the scores s of 32 KB keys (transposed, -infinity
    // where hidden); result and sum are rescaled if it has grown.
    template <int KB>
    __device__ __forceinline__ void grow(const f32x16 (&s)[KB], float c) {
        float mx = s[0][0];
#pragma unroll
        for (int e = 1; e < KB * 16; ++e) mx = fmaxf(mx, s[e >> 4][e & 15]);
        mx = pair_max(mx);
        if (__any((mx * c > mc + 8.0f) | (m == -INFINITY))) {
            const float m2 = fmaxf(m, mx);
            const float mc2 = m2 == -INFINITY ? 0.0f : m2 * c;
            const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mc - mc2);
            m = m2;
            mc = mc2;
            l *= f;
#pragma unroll
            for (int db = 0; db < DB; ++db) o[db] *= f;
        }
    }
    // The scores become weights.
    template <int KB>
    __device__ __forceinline__ void weights(f32x16 (&s)[KB], float c) {
#pragma unroll
        for (int e = 0; e < KB * 16; ++e) {
            const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e >> 4][e & 15], c, -mc));
            s[e >> 4][e & 15] = w;
            l += w;
        }
    }
    // The sum over both halves; false if no key was seen.
    __device__ __forceinline__ bool finish() {
        l = pair_sum(l);
        return (m != -INFINITY) | (l != 0.0f);
    }
    // The result becomes zero where `keep` is false; one test if none is.
    __device__ __forceinline__ void only(bool keep) { zero_unless<DB>(o, keep); }
};

__device__ __forceinline__ float log_sum(float mc, float l) {
    return (mc + __builtin_amdgcn_logf(l)) * kLn2;
}

// Forward.  A workgroup of 4 waves takes 128 rows (32 per wave) of one key
// head and walks the tiles of BN keys they see.  Per tile a wave forms
// S^T = K Q^T (keys in registers, its 32 rows across the lanes), so a row's
// maximum and sum are a lane's own registers plus one exchange with lane ^ 32,
// its factor is one value per lane, and the weights, rounded to the type (a
// product of 32-bit weights would run at an eighth of the rate; half a step of
// the type on weights of one sign), are already the operand of O^T += V^T P^T.
//
// Two tiles' buffers: the next tile is on its way (global memory to LDS, no
// registers) while this one is used.  At D = 128 the matrix cores bound it:
// 16k causal, 16 heads on 4, bfloat16: 1.17 ms, 1.03 PFLOP/s, 84 % of a large
// library product.  At D = 64 the vector unit does: a wave's 32 x 64 scores cost
// it about 1000 cycles (exponential, product, maximum, sum and rounding of
// each), the matrix cores half of that; a workgroup's sequence, its rows and
// first tile take another 6000 to 7000 cycles, more than the walk of a short
// event.  84k pulses, window 257, 8 heads on 2: 0.14 ms; 64 events of at most
// 128 tokens, 12 heads: 14 us (7 us of bytes).  A third buffer cost 5 %, scores
// formed one tile ahead 5 to 15 % (and spills at D = 128).
template <class T, int DP, int BN>
__global__ __launch_bounds__(256, 512 / (DP * (int)sizeof(T))) void attention_kernel(AttnArgs a) {
    constexpr int DB = DP / 32, STEPS = DP / 16;
    using Tl = Tile<T, DP>;
    using Frag = typename Elem<T>::Frag;
    __shared__ __attribute__((aligned(16))) char smem[2 * 2 * BN * Tl::kPitch];
    __shared__ BadRows bad;  // values taken out of tiles
    FPSTOK_LDS char* lds = (FPSTOK_LDS char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = a.G;
    RowTile t;
    if (!row_tile<7, false>(a, a.splits, t)) return;
    const QueryRows q(a, t, wave * 32, lane);
    Frag qf[STEPS];
    q.load<T, STEPS>(qf, a.q, a.D, half);
    const Window win(a, q.qi + t.tk - t.tq, t.tk);
    const bool wave_live = wave * 32 < t.rows;

    KeyTiles<BN> kt(a, q.pa, q.pb, t.tk);
    const int n = t.rows > 0 ? kt.part(t.part, a.splits) : 0;
    const T* kb = (const T*)a.k.data + t.k0 * a.k.row + t.hk * a.k.head;
    const T* vb = (const T*)a.v.data + t.k0 * a.v.row + t.hk * a.v.head;
    const Dma<T, DP, BN> dma(a.D, tid);
    const uint32_t off_k = dma.offset(a.k.row), off_v = dma.offset(a.v.row);
    // the tile loaded last and its keys
    int jn = n > 0 ? kt.tile(0) * BN : 0;
    const T* kp = kb + jn * a.k.row;
    const T* vp = vb + jn * a.v.row;
    auto load = [&](int i) {  // tile i on its way to its buffer; tiles in turn
        FPSTOK_LDS char* buf = lds + (i & 1) * 2 * BN * Tl::kPitch;
        if (i > 0) {
            const int skip = kt.from + i == kt.sink ? kt.first * BN - jn : BN;
            jn += skip;
            kp += skip * a.k.row;
            vp += skip * a.v.row;
        }
        dma.load(kp, off_k, a.k.row, t.tk - jn, buf, wave);
        dma.load(vp, off_v, a.v.row, t.tk - jn, buf + BN * Tl::kPitch, wave);
    };
    const View<BN> all(a, q.pa, q.pb, t.tk);
    const View<32> mine(a, q.wa, q.wb, t.tk);
    auto arrive = [&](int i) {  // this wave's part of it is there
        dma_wait();
        // a value that some row must not see meets a weight of 0 there: an
        // infinite one has to leave the product
        if (all.of(a, jn) == 1) {
            const uint32_t chunks = dma.clean(lds + ((i & 1) * 2 + 1) * BN * Tl::kPitch, tid);
#pragma unroll 1
            for (uint32_t c = chunks; c != 0; c &= c - 1)
                bad.note(i, __builtin_ctz(c) * dma.kStep + dma.row);
        }
    };

    Softmax<T, DB> sm;
    const float c = a.scale * kLog2e;
    constexpr int NB = DP == 64 || BN == 32 ? 1 : 2;
    // 32 NB keys (j0 on) from row `from` of the tile at kbuf on; v0, v1: what
    // the first and the second block of 32 look like (tile_view)
    auto attend = [&](const FPSTOK_LDS char* kbuf, int from, int j0, int v0, int v1) {
        const FPSTOK_LDS char* vbuf = kbuf + (BN + from) * Tl::kPitch;
        kbuf += from * Tl::kPitch;
        f32x16 s[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            f32x16 x = 0.0f;
#pragma unroll
            for (int st = 0; st < STEPS; ++st)
                if (sizeof(T) == 2 || st * 16 < a.D)  // (float32: a step is 8 instructions)
                    x = Elem<T>::mma(Tl::row_frag(kbuf, b * 32 + (lane & 31), st, half), qf[st], x);
            s[b] = x;
        }
        if (v0 != 2) win.mask(s[0], j0, half, a.sinks, -INFINITY);
        if (NB == 2 && v1 != 2) win.mask(s[NB - 1], j0 + 32, half, a.sinks, -INFINITY);
        sm.grow(s, c);
        sm.weights(s, c);
#pragma unroll
        for (int k = 0; k < NB * 2; ++k) {
            const Frag pf = to_frag<T>(s[k >> 1], k & 1);
#pragma unroll
            for (int db = 0; db < DB; ++db)
                if (sizeof(T) == 2 || db * 32 < a.D)
                    sm.o[db] = Elem<T>::mma(Tl::col_frag(vbuf, k * 16, db, lane), pf, sm.o[db]);
        }
    };
    bad.clear(tid);
    if (a.D < DP) dma.zero(lds, sizeof(smem), tid);
    __syncthreads();
    if (n > 0) {
        load(0);
        arrive(0);
    }
    __syncthreads();
    for (int i = 0; i < n; ++i) {
        const int j0 = jn;
        if (i + 1 < n) load(i + 1);
        const FPSTOK_LDS char* kbuf = lds + (i & 1) * 2 * BN * Tl::kPitch;
        // NB blocks of 32 keys at a time.  At D = 64 the walk is bound by the
        // vector unit: one block at a time skips blocks out of sight and leaves
        // registers for four workgroups per compute unit (two at a time: 84k-pulse
        // windows 184 us against 168).  At D = 128 two at a time keep the
        // matrix cores fed (one at a time: causal 16k 1.41 ms against 1.25).
        auto blocks = [&](int b) {
            const int v0 = wave_live ? mine.of(a, j0 + b) : 0;
            const int v1 = NB == 2 && wave_live ? mine.of(a, j0 + b + 32) : 0;
            if ((v0 | v1) != 0) attend(kbuf, b, j0 + b, v0, v1);
        };
        if constexpr (NB * 32 == BN)
            blocks(0);
        else
#pragma unroll 1
            for (int b = 0; b < BN; b += NB * 32) blocks(b);
        if (i + 1 < n) arrive(i + 1);
        __syncthreads();
    }
    const bool some = sm.finish();
    if (a.splits > 1) {
        const int64_t at =
            ((int64_t)t.part * a.Hk + t.hk) * a.qs.rows * G + t.q0 * G + t.row0 + q.r;
        float* part = a.part + at * a.D;
        sm.only(some);
        store_row<float, DB>(sm.o, 1.0f, q.live ? part : nullptr, a.D, lane);
        if (q.live && half == 0) a.part_ml[at] = make_float2(some ? sm.mc : -INFINITY, sm.l);
        if (bad.tiles != 0) {
            __syncthreads();
            add_bad_keys<BN>(part, a, kt, n, bad, q, t.tk, win, q.live, half, vb, a.v.row);
        }
        return;
    }
    const bool write = q.live || q.r < t.pad;
    T* out = (T*)a.out.data + q.row * a.out.row + q.h * a.out.head;
    sm.only(q.live && some);
    store_row<T, DB>(sm.o, q.live && some ? 1.0f / sm.l : 0.0f, write ? out : nullptr, a.D, lane);
    if (a.lse && half == 0 && write)
        a.lse[q.row * a.H + q.h] = !q.live ? 0.0f : some ? log_sum(sm.mc, sm.l) : -INFINITY;
    if (bad.tiles != 0) {
        __syncthreads();
        // (a row whose every score is -infinity stays 0)
        add_bad_keys<BN>(out, a, kt, n, bad, q, t.tk, win, q.live && some, half, vb, a.v.row);
    }
}

// Forward for sequences of at most 32 rows per key head (one query, or a few,
// against many keys): a workgroup takes 32 rows and its 4 waves take turns at
// the key tiles, each with its own LDS, running maximum and sum; they are
// joined at the end.  No wave waits for another inside the walk, so 4 tiles of
// K and V per workgroup are on their way at a time.  Bound by reading K and V
// once: 256 padded events of up to 1024 tokens, 12 heads, 84 us; 4 sequences of
// up to 131072 keys of 8 heads (32 query heads, D = 128), split, 170 us and 5 us
// for the join: 5.2 TB/s, a large copy's rate.  Tiles of 64 keys leave one
// workgroup per compute unit: 435 us there.  Sequences of more than 32 rows are
// slower here (64 events of up to 128 tokens: 30 us against 14), for every 32
// rows read all keys again.
template <class T, int DP, int BN>
__global__ __launch_bounds__(256, 512 / (DP * (int)sizeof(T)) > 3 ? 3 : 512 / (DP * (int)sizeof(T)))
void attention_few_kernel(AttnArgs a) {
    constexpr int BM = 32, DB = DP / 32, KB = BN / 32, STEPS = DP / 16;
    using f4 = float __attribute__((ext_vector_type(4)));
    using Tl = Tile<T, DP>;
    using Frag = typename Elem<T>::Frag;
    constexpr int kWaveBytes = 2 * BN * Tl::kPitch;
    // the join keeps 32 x DP floats of every wave in its tiles' place
    static_assert(kWaveBytes >= BM * DP * 4, "join buffer");
    __shared__ __attribute__((aligned(16))) char smem[4 * kWaveBytes];
    __shared__ float2 ml[4][BM];
    __shared__ BadRows bad;
    FPSTOK_LDS char* lds = (FPSTOK_LDS char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = a.G;
    RowTile t;
    if (!row_tile<5, false>(a, a.splits, t)) return;
    const QueryRows q(a, t, 0, lane);
    Frag qf[STEPS];
    q.load<T, STEPS>(qf, a.q, a.D, half);
    const Window win(a, q.qi + t.tk - t.tq, t.tk);

    KeyTiles<BN> kt(a, q.pa, q.pb, t.tk);
    const int n = t.rows > 0 ? kt.part(t.part, a.splits) : 0;
    const T* kb = (const T*)a.k.data + t.k0 * a.k.row + t.hk * a.k.head;
    const T* vb = (const T*)a.v.data + t.k0 * a.v.row + t.hk * a.v.head;
    Stage<T, DP, BN, 64> sk, sv;
    FPSTOK_LDS char* kbuf = lds + wave * kWaveBytes;
    FPSTOK_LDS char* vbuf = kbuf + BN * Tl::kPitch;
    auto load = [&](int i) {
        const int64_t j0 = (int64_t)kt.tile(i) * BN;
        sk.load(kb + j0 * a.k.row, a.k.row, t.tk - (int)j0, a.D, lane);
        sv.load(vb + j0 * a.v.row, a.v.row, t.tk - (int)j0, a.D, lane);
    };

    const View<BN> all(a, q.pa, q.pb, t.tk);
    Softmax<T, DB> sm;
    const float c = a.scale * kLog2e;
    if (wave < n) load(wave);
    bad.clear(tid);
    __syncthreads();
    for (int i = wave; i < n; i += 4) {
        const int j0 = kt.tile(i) * BN;
        const int view = all.of(a, j0);
        if (view == 1) {
            const uint32_t chunks = sv.clean(lane);
#pragma unroll 1
            for (uint32_t c = chunks; c != 0; c &= c - 1)
                bad.note(i, __builtin_ctz(c) * sv.kStep + sv.row(lane));
        }
        wave_sync();  // the wave's reads of the last tile are done
        sk.store(kbuf, a.D, lane);
        sv.store(vbuf, a.D, lane);
        wave_sync();
        if (i + 4 < n) load(i + 4);
        f32x16 s[KB];
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            f32x16 x = 0.0f;
#pragma unroll
            for (int st = 0; st < STEPS; ++st)
                if (sizeof(T) == 2 || st * 16 < a.D)  // (float32: a step is 8 instructions)
                    x = Elem<T>::mma(Tl::row_frag(kbuf, b * 32 + (lane & 31), st, half), qf[st], x);
            s[b] = x;
        }
        if (view == 1) {
#pragma unroll
            for (int b = 0; b < KB; ++b)
                win.mask(s[b], j0 + b * 32, half, a.sinks, -INFINITY);
        }
        sm.grow(s, c);
        sm.weights(s, c);
#pragma unroll
        for (int k = 0; k < KB * 2; ++k) {
            const Frag pf = to_frag<T>(s[k >> 1], k & 1);
#pragma unroll
            for (int db = 0; db < DB; ++db)
                if (sizeof(T) == 2 || db * 32 < a.D)
                    sm.o[db] = Elem<T>::mma(Tl::col_frag(vbuf, k * 16, db, lane), pf, sm.o[db]);
        }
    }
    const bool seen = sm.finish();
    sm.only(seen);
    wave_sync();
    if (half == 0) ml[wave][q.r] = make_float2(seen ? sm.mc : -INFINITY, sm.l);
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            f4 x;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = sm.o[db][g * 4 + e];
            *(FPSTOK_LDS f4*)(kbuf + (q.r * DP + db * 32 + g * 8 + half * 4) * 4) = x;
        }
    __syncthreads();
    // 4 elements per thread and turn
    const int64_t part0 =
        ((int64_t)t.part * a.Hk + t.hk) * a.qs.rows * G + t.q0 * G + t.row0;
    const int rows = t.rows > t.pad ? t.rows : t.pad;
    for (int x = tid; x < rows * (DP / 4); x += 256) {
        const int row = x / (DP / 4), d = (x % (DP / 4)) * 4;
        if (d >= a.D) continue;
        const int qi = (t.row0 + row) / G, h = t.hk * G + (t.row0 + row) - qi * G;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) top = fmaxf(top, ml[w][row].x);
        float sum = 0.0f;
        f4 y = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float2 z = ml[w][row];
            const float f = z.x == -INFINITY && z.y == 0.0f ? 0.0f
                                                              : __builtin_amdgcn_exp2f(z.x - top);
            sum += z.y * f;
            y += f * *(FPSTOK_LDS f4*)(lds + w * kWaveBytes + (row * DP + d) * 4);
        }
        const bool here = row < t.rows, some = top != -INFINITY || sum != 0.0f;
        if (a.splits > 1) {
            if (!here) continue;
            *(f4*)(a.part + (part0 + row) * a.D + d) = y;
            if (d == 0) a.part_ml[part0 + row] = make_float2(some ? top : -INFINITY, sum);
            continue;
        }
        y *= here && some ? 1.0f / sum : 0.0f;
        if (!here || !some) y = 0.0f;
        using T4 = T __attribute__((ext_vector_type(4)));
        *(T4*)((T*)a.out.data + (t.q0 + qi) * a.out.row + h * a.out.head + d) =
            __builtin_convertvector(y, T4);
        if (a.lse && d == 0)
            a.lse[(t.q0 + qi) * a.H + h] = !here ? 0.0f : some ? log_sum(top, sum) : -INFINITY;
    }
    if (bad.tiles != 0) {
        __syncthreads();
        if (wave == 0) {
            bool some = false;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                some |= !(ml[w][q.r].x == -INFINITY && ml[w][q.r].y == 0.0f);
            if (a.splits > 1)
                add_bad_keys<BN>(a.part + (part0 + q.r) * a.D, a, kt, n, bad, q, t.tk, win,
                                     q.live, half, vb, a.v.row);
            else  // (a row whose every score is -infinity stays 0)
                add_bad_keys<BN>((T*)a.out.data + q.row * a.out.row + q.h * a.out.head, a, kt,
                                     n, bad, q, t.tk, win, q.live && some, half, vb, a.v.row);
        }
    }
}

// Joins the parts of a row whose keys were split: a workgroup per (query,
// head).  Its threads take 4 elements each of every kGroups-th part, so a
// thread's loads do not wait for one another; the groups' sums are added in
// order.
template <class T>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a) {
    using f4 = float __attribute__((ext_vector_type(4)));
    constexpr int kGroups = 8;
    __shared__ float factor[256];  // at most 256 parts
    __shared__ f4 sums[kGroups][32];
    __shared__ float wave_top[4], wave_sum[4];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t row = blockIdx.x / a.H;
    const int h = (int)(blockIdx.x % a.H), G = a.G, hk = h / G;
    bool here = true;
    if (a.qs.cu) {
        if (row < cu_at(a.qs, 0) || row >= cu_at(a.qs, a.qs.B)) return;
    } else {
        here = row % a.qs.cap < a.qs.count[row / a.qs.cap];
    }
    const int64_t step = (int64_t)a.Hk * a.qs.rows * G;
    const int64_t at = ((int64_t)hk * a.qs.rows + row) * G + h - hk * G;
    float2 z = make_float2(-INFINITY, 0.0f);
    if (here && tid < a.splits) z = a.part_ml[tid * step + at];
    const bool seen = !(z.x == -INFINITY && z.y == 0.0f);
    float top = z.x;
#pragma unroll
    for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    if (lane == 0) wave_top[tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(wave_top[0], wave_top[1]), fmaxf(wave_top[2], wave_top[3]));
    const float f = seen ? __builtin_amdgcn_exp2f(z.x - top) : 0.0f;
    factor[tid] = f;
    float sum = z.y * f;
#pragma unroll
    for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
    if (lane == 0) wave_sum[tid >> 6] = sum;
    __syncthreads();
    sum = (wave_sum[0] + wave_sum[1]) + (wave_sum[2] + wave_sum[3]);
    const int d = (tid & 31) * 4, group = tid >> 5;
    if (here) {
        f4 y = 0.0f;
        const float* part = a.part + at * a.D + (d < a.D ? d : 0);
        const int64_t stride = step * a.D;
#pragma unroll 4
        for (int s = group; s < a.splits; s += kGroups)
            y += factor[s] * *(const f4*)(part + s * stride);
        sums[group][tid & 31] = y;
    }
    __syncthreads();
    const bool some = here && (top != -INFINITY || sum != 0.0f);
    if (tid < 32 && d < a.D) {
        f4 y = 0.0f;
        if (some) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g) y += sums[g][tid];
            y *= 1.0f / sum;
        }
        using T4 = T __attribute__((ext_vector_type(4)));
        *(T4*)((T*)a.out.data + row * a.out.row + h * a.out.head + d) =
            __builtin_convertvector(y, T4);
    }
    if (a.lse && tid == 0)
        a.lse[row * a.H + h] =
            !here ? 0.0f
                  : some ? (top + __builtin_amdgcn_logf(sum)) * 0.693147180559945f : -INFINITY;
}

// The same for many rows: 4 elements of one (query, head) per thread, its parts
// one after the other.
template <class T>
__global__ __launch_bounds__(256) void attention_join_rows_kernel(AttnArgs a) {
    using f4 = float __attribute__((ext_vector_type(4)));
    using T4 = T __attribute__((ext_vector_type(4)));
    const uint32_t per = (uint32_t)a.D / 4;
    const uint32_t x = blockIdx.x * 256u + threadIdx.x;
    const uint32_t rh = x / per;
    const int d = (int)(x - rh * per) * 4;
    const uint32_t row = rh / (uint32_t)a.H;
    if (row >= a.qs.rows) return;
    const int h = (int)(rh - row * (uint32_t)a.H), hk = h / a.G;
    bool here = true;
    if (a.qs.cu) {
        if (row < cu_at(a.qs, 0) || row >= cu_at(a.qs, a.qs.B)) return;
    } else {
        const uint32_t b = row / (uint32_t)a.qs.cap;
        here = (int)(row - b * (uint32_t)a.qs.cap) < a.qs.count[b];
    }
    const int64_t step = (int64_t)a.Hk * a.qs.rows * a.G;
    const int64_t at = ((int64_t)hk * a.qs.rows + row) * a.G + h - hk * a.G;
    float top = -INFINITY, sum = 0.0f;
    f4 y = 0.0f;
    if (here) {
#pragma unroll 4
        for (int s = 0; s < a.splits; ++s) top = fmaxf(top, a.part_ml[s * step + at].x);
#pragma unroll 4
        for (int s = 0; s < a.splits; ++s) {
            const float2 z = a.part_ml[s * step + at];
            const float f =
                z.x == -INFINITY && z.y == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(z.x - top);
            sum += z.y * f;
            y += f * *(const f4*)(a.part + (s * step + at) * a.D + d);
        }
    }
    const bool some = here && (top != -INFINITY || sum != 0.0f);
    y *= some ? 1.0f / sum : 0.0f;
    if (!some) y = 0.0f;
    *(T4*)((T*)a.out.data + row * a.out.row + h * a.out.head + d) = __builtin_convertvector(y, T4);
    if (a.lse && d == 0)
        a.lse[(int64_t)row * a.H + h] = !here ? 0.0f : some ? log_sum(top, sum) : -INFINITY;
}

// grad_q, and the rows' statistics for the kernel below.  Rows and key tiles as
// in the forward kernel; per 32 keys a wave forms S^T = K Q^T and
// dP^T = V dO^T, and dS^T = P^T (dP^T - delta), rounded to the type, is the
// operand of dQ^T += K^T dS^T.
//
// delta = grad_out times the rounded out is off by that rounding, and in rows
// of few keys this is a large part of grad_q's and grad_k's error (8 keys of
// bfloat16: 1.57 times the error of rounding the exact gradient, 1.42 without;
// 64 keys: 1.45 and 1.43).  dS summed over the keys, which should be 0, gives the
// difference to the exact delta: where one tile is all a row tile sees it is
// formed from that tile first, and with a window of fewer than 32 keys (TWICE)
// the whole walk is made twice (at 256 events of up to 256 tokens this is 3 % of
// the backward pass).  It goes by tiles, so the first rows of a long causal
// sequence, which see few keys in a row tile that sees two key tiles, keep the
// larger error.
//
// 3 products where 2 are the gradient's own: forming S and dP here and again
// for grad_k and grad_v costs 2 of 7, and adding one kernel's grad_q up over the
// workgroups of a sequence's keys would cost a float32 result per workgroup, or
// atomics whose order changes it.  6000 + 2111 + 64 rows, 16 heads on 8, D =
// 128, bfloat16: 0.48 ms, 1.04 PFLOP/s; 256 events of up to 256 tokens, 12
// heads, D = 64: 117 us.
//
// A tile that some row does not see whole loses its infinite elements of K.  A
// key that lost some has no finite score: in a row that sees it the score is
// -infinity and the weight 0, or the row's lse is not a number and with it
// its whole gradient.  So the scores of such keys are set to -infinity, and 0
// times the lost element, which is not a number, is added after the walk.
template <class T, int DP, int BN, bool TWICE>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void attention_dq_kernel(AttnArgs a) {
    constexpr int DB = DP / 32, KB = BN / 32, STEPS = DP / 16;
    using Tl = Tile<T, DP>;
    using Frag = typename Elem<T>::Frag;
    __shared__ __attribute__((aligned(16))) char smem[2 * 2 * BN * Tl::kPitch];
    __shared__ BadRows bad;
    __shared__ int lost[2][BN];  // of a buffer's keys: 1 + the tile in which one lost elements
    FPSTOK_LDS char* lds = (FPSTOK_LDS char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    RowTile t;
    if (!row_tile<7, false>(a, 1, t)) return;
    const QueryRows q(a, t, wave * 32, lane);
    const Window win(a, q.qi + t.tk - t.tq, t.tk);
    const bool wave_live = wave * 32 < t.rows;
    Frag qf[STEPS], gf[STEPS], of[STEPS];
    q.load<T, STEPS>(qf, a.q, a.D, half);
    q.load<T, STEPS>(gf, a.grad_out, a.D, half);
    q.load<T, STEPS>(of, a.out, a.D, half);
    const float lse = q.live ? a.lse[q.row * a.H + q.h] : 0.0f;

    KeyTiles<BN> kt(a, q.pa, q.pb, t.tk);
    const int n = t.rows > 0 ? kt.count : 0;
    const T* kb = (const T*)a.k.data + t.k0 * a.k.row + t.hk * a.k.head;
    const T* vb = (const T*)a.v.data + t.k0 * a.v.row + t.hk * a.v.head;
    const Dma<T, DP, BN> dma(a.D, tid);
    const uint32_t off_k = dma.offset(a.k.row), off_v = dma.offset(a.v.row);
    // the tile loaded last and its keys
    int jn = n > 0 ? kt.tile(0) * BN : 0;
    const T* kp = kb + jn * a.k.row;
    const T* vp = vb + jn * a.v.row;
    auto load = [&](int i) {  // tile i on its way to its buffer; tiles in turn
        FPSTOK_LDS char* buf = lds + (i & 1) * 2 * BN * Tl::kPitch;
        if (i > 0) {
            const int skip = kt.from + i == kt.sink ? kt.first * BN - jn : BN;
            jn += skip;
            kp += skip * a.k.row;
            vp += skip * a.v.row;
        }
        dma.load(kp, off_k, a.k.row, t.tk - jn, buf, wave);
        dma.load(vp, off_v, a.v.row, t.tk - jn, buf + BN * Tl::kPitch, wave);
    };
    const View<BN> all(a, q.pa, q.pb, t.tk);
    const View<32> mine(a, q.wa, q.wb, t.tk);
    auto arrive = [&](int i) {
        dma_wait();
        if (all.of(a, jn) != 1) return;
        FPSTOK_LDS char* buf = lds + (i & 1) * 2 * BN * Tl::kPitch;
        const uint32_t chunks = dma.clean(buf, tid);
#pragma unroll 1
        for (uint32_t c = chunks; c != 0; c &= c - 1) {
            const int row = __builtin_ctz(c) * dma.kStep + dma.row;
            bad.note(i, row);
            lost[i & 1][row] = i + 1;
        }
    };

    f32x16 dq[DB];
#pragma unroll
    for (int db = 0; db < DB; ++db) dq[db] = 0.0f;
    const float c = a.scale * kLog2e;
    float delta = 0.0f, lse2 = 0.0f;
    // tile i may hold keys that lost elements
    auto lost_in = [&](int i) { return __builtin_amdgcn_readfirstlane(bad.tiles) >> (i & 31) & 1; };
    // the scores of such keys, of 32 from row b of tile i on
    auto hide_lost = [&](f32x16& x, int b, int i) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            x[e] = lost[i & 1][b + (e >> 2) * 8 + half * 4 + (e & 3)] == i + 1 ? -INFINITY : x[e];
    };
    // sum of dS over the keys of 32 rows from row b of the tile at kbuf on
    auto add_delta = [&](const FPSTOK_LDS char* kbuf, int b, int j0, bool mask, bool holes, int i,
                         float& sum) {
        f32x16 x = 0.0f, y = 0.0f;
#pragma unroll
        for (int st = 0; st < STEPS; ++st) {
            const int row = b + (lane & 31);
            x = Elem<T>::mma(Tl::row_frag(kbuf, row, st, half), qf[st], x);
            y = Elem<T>::mma(Tl::row_frag(kbuf + BN * Tl::kPitch, row, st, half), gf[st], y);
        }
        if (holes) hide_lost(x, b, i);
#pragma unroll
        for (int e = 0; e < 16; ++e)
            x[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[e], c, -lse2)) * (y[e] - delta);
        if (mask) win.mask(x, j0 + b, half, a.sinks, 0.0f);
#pragma unroll
        for (int e = 0; e < 16; ++e) sum += x[e];
    };
    auto block = [&](const FPSTOK_LDS char* kbuf, int b, int j0, bool mask, bool holes, int i) {
        const FPSTOK_LDS char* vbuf = kbuf + BN * Tl::kPitch;
        f32x16 x = 0.0f, y = 0.0f;
#pragma unroll
        for (int st = 0; st < STEPS; ++st) {
            x = Elem<T>::mma(Tl::row_frag(kbuf, b * 32 + (lane & 31), st, half), qf[st], x);
            y = Elem<T>::mma(Tl::row_frag(vbuf, b * 32 + (lane & 31), st, half), gf[st], y);
        }
        if (holes) hide_lost(x, b * 32, i);
        f32x16 ds;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            ds[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[e], c, -lse2)) * (y[e] - delta);
        if (mask) win.mask(ds, j0 + b * 32, half, a.sinks, 0.0f);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const Frag f = to_frag<T>(ds, k);
#pragma unroll
            for (int db = 0; db < DB; ++db)
                dq[db] = Elem<T>::mma(Tl::col_frag(kbuf, b * 32 + k * 16, db, lane), f, dq[db]);
        }
    };
    bad.clear(tid);
    if (tid < 2 * BN) lost[tid / BN][tid % BN] = 0;
    if (a.D < DP) dma.zero(lds, sizeof(smem), tid);
    __syncthreads();
    if (n > 0) load(0);
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) delta = __builtin_fmaf((float)gf[s][e], (float)of[s][e], delta);
    // a row that sees nothing, or nothing but scores of -infinity: its weights
    // are exp2(score - infinity) = 0, here and for grad_k and grad_v
    const bool some = lse != -INFINITY;
    delta = some ? pair_sum(delta) : 0.0f;
    lse2 = some ? lse * kLog2e : INFINITY;
    if (n > 0) arrive(0);
    __syncthreads();
    float off_by = 0.0f;
    if (!TWICE && sizeof(T) == 2 && n == 1 && wave_live) {
#pragma unroll 1
        for (int b = 0; b < BN; b += 32) {
            const int view = mine.of(a, jn + b);
            if (view != 0) add_delta(lds, b, jn, view == 1, lost_in(0), 0, off_by);
        }
        delta += pair_sum(off_by);
    }
    if constexpr (TWICE) {
        for (int i = 0; i < n; ++i) {
            const int j0 = jn;
            if (i + 1 < n) load(i + 1);
            const bool holes = lost_in(i);
#pragma unroll 1
            for (int b = 0; b < BN; b += 32) {
                const int view = wave_live ? mine.of(a, j0 + b) : 0;
                if (view != 0)
                    add_delta(lds + (i & 1) * 2 * BN * Tl::kPitch, b, j0, view == 1, holes, i,
                              off_by);
            }
            if (i + 1 < n) arrive(i + 1);
            __syncthreads();
        }
        delta += pair_sum(off_by);
        jn = n > 0 ? kt.tile(0) * BN : 0;
        kp = kb + jn * a.k.row;
        vp = vb + jn * a.v.row;
        if (n > 0) {
            load(0);
            arrive(0);
        }
        __syncthreads();
    }
    if (q.live && half == 0) {
        const int64_t at = (int64_t)q.h * a.qs.rows + q.row;
        a.lse2[at] = lse2;
        a.delta[at] = some ? delta : 0.0f;
    }
    for (int i = 0; i < n; ++i) {
        const int j0 = jn;
        if (i + 1 < n) load(i + 1);
        const FPSTOK_LDS char* kbuf = lds + (i & 1) * 2 * BN * Tl::kPitch;
        const bool holes = lost_in(i);
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            const int view = wave_live ? mine.of(a, j0 + b * 32) : 0;
            if (view != 0) block(kbuf, b, j0, view == 1, holes, i);
        }
        if (i + 1 < n) arrive(i + 1);
        __syncthreads();
    }
    T* out = (T*)a.grad_q.data + q.row * a.grad_q.row + q.h * a.grad_q.head;
    zero_unless<DB>(dq, q.live && some);
    store_row<T, DB>(dq, a.scale, q.live || q.r < t.pad ? out : nullptr, a.D, lane);
    if (bad.tiles != 0) {
        __syncthreads();
        add_bad_keys<BN, true>(out, a, kt, n, bad, q, t.tk, win, q.live && some, half, kb,
                                   a.k.row);
    }
}

// The last query that sees a sequence's first key tile (128 keys, the sinks
// among them) through the window, -1 if none does; later ones see its sinks
// only.
__device__ __forceinline__ int last_by_window(const AttnArgs& a, int tq, int tk) {
    const int jl = (tk < 128 ? tk : 128) - 1, i1 = jl + a.left - (tk - tq);
    return i1 < -1 ? -1 : i1 < tq - 1 ? i1 : tq - 1;
}

// The sinks' gradients from the rows that see nothing else of the first key
// tile: in a long sequence that is nearly every row, and one workgroup walking
// them all would take longer than everything else.  A workgroup takes a chunk
// of them, its waves 32 rows in turn; nothing is masked.  Rows without weights,
// and rows past the last one, have lse2 = infinity (see below).  The chunks' parts
// are added in order by the kernel below.  (40k + 12k + 2.5k pulses, 4 sinks, 8
// heads on 4: the walk in one workgroup 4 ms, in chunks 27 us.  At float32 and
// D > 64 its two results and two operands pass the registers and spill.)
template <class T, int DP>
__global__ __launch_bounds__(256, DP * (int)sizeof(T) <= 128 ? 2 : 1)
void attention_sink_kernel(AttnArgs a) {
    constexpr int DB = DP / 32, STEPS = DP / 16;
    using f4 = float __attribute__((ext_vector_type(4)));
    using Tl = Tile<T, DP>;
    using Frag = typename Elem<T>::Frag;
    constexpr int kTile = 32 * Tl::kPitch;
    // 32 x DP floats of a wave's result in its tiles' place
    constexpr int kWaveBytes = 2 * kTile > 32 * DP * 4 ? 2 * kTile : 32 * DP * 4;
    __shared__ __attribute__((aligned(16))) char smem[4 * kWaveBytes];
    __shared__ __attribute__((aligned(16))) float stat[4][2][32];
    FPSTOK_LDS char* lds = (FPSTOK_LDS char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = a.G, hk = (int)(blockIdx.x % (uint32_t)a.Hk);
    const uint32_t slot = blockIdx.x / (uint32_t)a.Hk;
    const int chunk = 1 << a.sink_shift;
    int64_t q0, k0, c;
    int tq, tk, b;
    if (a.qs.cu) {
        b = find_seq(a.qs, slot, 1, a.sink_shift, q0, tq, c);
    } else {
        const uint32_t per = (uint32_t)((a.qs.cap + chunk - 1) >> a.sink_shift);
        b = (int)(slot / per);
        c = slot % per;
        seq_rows(a.qs, b, q0, tq);
    }
    seq_rows(a.ks, b, k0, tk);
    if (c < 0 || tq == 0 || tk == 0) return;
    const int i0 = last_by_window(a, tq, tk) + 1;
    const int64_t from = c << a.sink_shift;
    if (from >= tq - i0) return;
    const int left = tq - i0 - (int)from, rows = left < chunk ? left : chunk;
    const int sinks = a.sinks < tk ? a.sinks : tk;
    // the chunk's first query, in head 0 of the group
    const int64_t row0 = q0 + i0 + from;
    const T* qb = (const T*)a.q.data + row0 * a.q.row + (int64_t)hk * G * a.q.head;
    const T* gb = (const T*)a.grad_out.data + row0 * a.grad_out.row +
                  (int64_t)hk * G * a.grad_out.head;
    FPSTOK_LDS char* qbuf = lds + wave * kWaveBytes;
    FPSTOK_LDS char* gbuf = qbuf + kTile;
    const float cs = a.scale * kLog2e;

    for (int s0 = 0; s0 < sinks; s0 += 32) {
        const int j = s0 + (lane & 31);
        const bool live = j < sinks;
        Frag kf[STEPS], vf[STEPS];
        load_row<T, STEPS>(kf, (const T*)a.k.data + (k0 + j) * a.k.row + hk * a.k.head, live,
                           (const T*)a.k.data, a.D, half);
        load_row<T, STEPS>(vf, (const T*)a.v.data + (k0 + j) * a.v.row + hk * a.v.head, live,
                           (const T*)a.v.data, a.D, half);
        f32x16 dk[DB], dv[DB];
#pragma unroll
        for (int db = 0; db < DB; ++db) dk[db] = 0.0f, dv[db] = 0.0f;
        Stage<T, DP, 32, 64> sq, sg;
        float2 st = make_float2(0.0f, 0.0f);
        auto load = [&](int g, int x) {  // 32 queries from x on, head g of the group
            sq.load(qb + x * a.q.row + g * a.q.head, a.q.row, rows - x, a.D, lane);
            sg.load(gb + x * a.grad_out.row + g * a.grad_out.head, a.grad_out.row, rows - x, a.D,
                    lane);
            const int r = lane & 31, last = rows - x - 1;
            const int64_t at = (int64_t)(hk * G + g) * a.qs.rows + row0 + x + (r < last ? r : last);
            st = make_float2(a.lse2[at], a.delta[at]);
            if (r > last) st = make_float2(INFINITY, 0.0f);
        };
        if (wave * 32 < rows) load(0, wave * 32);
        for (int g = 0, x = wave * 32; g < G && x < rows;) {
            wave_sync();  // the wave's reads of the last tile are done
            const uint32_t gone = (uint32_t)__ballot(st.x == INFINITY);
            if (gone != 0) {
                sq.have = 32;  // (rows past the last one are copies of it)
                sq.finite(gone, lane);
                sg.drop(gone, lane);
#pragma unroll
                for (int e = 0; e < STEPS; ++e) vf[e] = frag_clean<T>(vf[e]);
            }
            sq.store(qbuf, a.D, lane);
            sg.store(gbuf, a.D, lane);
            if (half == 0) stat[wave][0][lane] = st.x, stat[wave][1][lane] = st.y;
            wave_sync();
            x += 128;
            if (x >= rows) x = wave * 32, ++g;
            if (g < G) load(g, x);
            f32x16 s = 0.0f, y = 0.0f;
#pragma unroll
            for (int e = 0; e < STEPS; ++e) {
                s = Elem<T>::mma(Tl::row_frag(qbuf, lane & 31, e, half), kf[e], s);
                y = Elem<T>::mma(Tl::row_frag(gbuf, lane & 31, e, half), vf[e], y);
            }
            f32x16 w, ds;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int at = (e >> 2) * 8 + half * 4 + (e & 3);
                w[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], cs, -stat[wave][0][at]));
                ds[e] = w[e] * (y[e] - stat[wave][1][at]);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const Frag fw = to_frag<T>(w, e), fs = to_frag<T>(ds, e);
#pragma unroll
                for (int db = 0; db < DB; ++db) {
                    dv[db] = Elem<T>::mma(Tl::col_frag(gbuf, e * 16, db, lane), fw, dv[db]);
                    dk[db] = Elem<T>::mma(Tl::col_frag(qbuf, e * 16, db, lane), fs, dk[db]);
                }
            }
        }
        // the waves' results, added in order: [key][DP] floats in LDS
        float* part = a.sink_part + (((int64_t)slot * a.Hk + hk) * 2 * a.sinks + s0) * a.D;
        const int keys = sinks - s0 < 32 ? sinks - s0 : 32;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    f4 x;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[e] = which ? dv[db][g * 4 + e] : dk[db][g * 4 + e];
                    *(FPSTOK_LDS f4*)(qbuf + ((lane & 31) * DP + db * 32 + g * 8 + half * 4) * 4) =
                        x;
                }
            __syncthreads();
            for (int x = tid; x < keys * (DP / 4); x += 256) {
                const int key = x / (DP / 4), d = (x % (DP / 4)) * 4;
                if (d >= a.D) continue;
                f4 y = 0.0f;
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    y += *(FPSTOK_LDS f4*)(lds + w * kWaveBytes + (key * DP + d) * 4);
                *(f4*)(part + (int64_t)which * a.sinks * a.D + key * a.D + d) = y;
            }
        }
        __syncthreads();
    }
}

// Where part `split` of a key's gradients lies: [split][grad_k, grad_v][Hk][row].
__device__ __forceinline__ int64_t k_part_at(const AttnArgs& a, int split, int hk, int64_t row) {
    return (((int64_t)split * 2 * a.Hk + hk) * a.ks.rows + row) * a.D;
}

// grad_k and grad_v.  A workgroup takes 128 keys of one key head (32 per wave,
// across the lanes) and walks the queries that see them, BQ at a time, head
// after head of the group: S = Q K^T and dP = dO V^T have the rows in registers, so P
// and dS = P (dP - delta), rounded to the type, are the operands of
// dV^T += dO^T P and dK^T += Q^T dS.  The gradients of the group's heads add up
// in the accumulators, in a fixed order.  Where that leaves few workgroups (few
// keys, many queries or heads) the walk is split over several, whose parts are
// added by the kernel below.  4 products: 6000 + 2111 + 64 rows, D = 128: 0.74 ms,
// 0.90 PFLOP/s (V's operands from LDS, for its registers hold accumulators); at
// D = 64 the vector unit bounds it: 256 events of up to 256 tokens, 149 us.
//
// A query whose every visible score is -infinity adds nothing: its lse2 is
// infinity, so its weights exp2(score - infinity) are 0 as long as its scores
// stay below infinity and nothing they multiply is infinite.  A tile with such
// queries keeps the signs of their infinite elements only (1 in their place: a
// term of a score that was -infinity stays so, or is finite) and takes 0 for
// their gradient and for infinite values (any other query that sees one of those has
// a delta that is not finite).
template <class T, int DP, int BQ>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1)
void attention_dkv_kernel(AttnArgs a) {
    constexpr int DB = DP / 32, QB = BQ / 32, STEPS = DP / 16;
    using Tl = Tile<T, DP>;
    using Frag = typename Elem<T>::Frag;
    // at DP = 128 of a 16-bit type the accumulators leave no registers for V:
    // it is read from LDS
    constexpr bool kVLds = DP > 64 && sizeof(T) == 2;
    constexpr int kV = 2 * 2 * BQ * Tl::kPitch;
    __shared__ __attribute__((aligned(16))) char smem[kV + (kVLds ? 128 * Tl::kPitch : 0)];
    __shared__ __attribute__((aligned(16))) float stat[2][2][64];
    __shared__ BadRows bad;
    FPSTOK_LDS char* lds = (FPSTOK_LDS char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = a.G;
    RowTile t;
    if (!row_tile<7, true>(a, a.k_splits, t)) return;

    const int r = wave * 32 + (lane & 31);
    const bool live = r < t.rows;
    const int64_t krow = t.k0 + t.row0 + r;
    Frag kf[STEPS], vf[STEPS];
    load_row<T, STEPS>(kf, (const T*)a.k.data + krow * a.k.row + t.hk * a.k.head, live,
                       (const T*)a.k.data, a.D, half);
    if constexpr (!kVLds)
        load_row<T, STEPS>(vf, (const T*)a.v.data + krow * a.v.row + t.hk * a.v.head, live,
                           (const T*)a.v.data, a.D, half);
    // queries i0 .. i1 see some key of the tile (of the rows past its window,
    // the tile with the sinks gets their gradients from the kernel above), e0 ..
    // e1 of them this lane's key
    const int off = t.tk - t.tq, j = t.row0 + r;
    const int j_last = t.row0 + t.rows - 1;
    int i0 = 0, i1 = t.tq - 1, e0 = 0, e1;
    if (a.right >= 0 && t.row0 - a.right - off > 0) i0 = t.row0 - a.right - off;
    if (a.left >= 0 && j_last + a.left - off < i1) i1 = j_last + a.left - off;
    if (a.right >= 0 && j - a.right - off > 0) e0 = j - a.right - off;
    e1 = a.left >= 0 && j >= a.sinks && j + a.left - off < i1 ? j + a.left - off : i1;
    uint32_t e_span = (uint32_t)(e1 - e0);
    if (e1 < e0) e0 = 0x7fffffff, e_span = 0;  // none: no query has that number
    const int nq = t.rows > 0 && i1 >= i0 ? i1 - i0 + 1 : 0;
    // this workgroup's tiles of the walk: [from, from + n) of per tiles a head
    const int per = (nq + BQ - 1) / BQ, walk = per * G;
    int from = 0, n = walk;
    if (a.k_splits > 1) {
        const int each = (int)(((uint32_t)walk + (uint32_t)a.k_splits - 1) / (uint32_t)a.k_splits);
        from = t.part * each < walk ? t.part * each : walk;
        n = walk - from < each ? walk - from : each;
    }
    // `rows` (all_range) or 32 (any_range) queries from x on: x - lo <= span if
    // each of them exists and sees each of the keys j0 .. j1, or if some may see
    // some
    struct Range {
        int lo;
        uint32_t span;
        __device__ __forceinline__ Range(int a, int b) : lo(a), span((uint32_t)(b - a)) {
            if (b < a) lo = 0x7fffffff, span = 0;
        }
        __device__ __forceinline__ bool has(int x) const { return (uint32_t)(x - lo) <= span; }
    };
    auto all_range = [&](int j0, int j1, int rows) {
        const int lo = a.right >= 0 && j1 - a.right - off > 0 ? j1 - a.right - off : 0;
        int hi = i1;
        if (a.left >= 0 && j1 >= a.sinks && j0 + a.left - off < hi) hi = j0 + a.left - off;
        return Range(lo, hi - (rows - 1));
    };
    auto any_range = [&](int j0, int j1) {
        const int lo = a.right >= 0 ? j0 - a.right - off - 31 : 0;
        int hi = i1;
        if (a.left >= 0 && j0 >= a.sinks && j1 + a.left - off < hi) hi = j1 + a.left - off;
        return Range(lo < 0 ? 0 : lo, hi);
    };
    const int wj0 = t.row0 + wave * 32, wj1 = wj0 + 31 < j_last ? wj0 + 31 : j_last;
    const Range wave_all = all_range(wj0, wj1, 32), wave_any = any_range(wj0, wj1);
    const Range tile_all = all_range(t.row0, j_last, BQ);
    const bool wave_live = wave * 32 < t.rows;

    const Dma<T, DP, BQ> dma(a.D, tid);
    const uint32_t off_q = dma.offset(a.q.row), off_g = dma.offset(a.grad_out.row);
    // the first query of the tile loaded last, and where it lies
    const int head0 = n > 0 ? from / per : 0;
    int xn = i0 + (n > 0 ? from - head0 * per : 0) * BQ;
    const int64_t row_n = t.q0 + xn, head_n = (int64_t)t.hk * G + head0;
    const T* qp = (const T*)a.q.data + row_n * a.q.row + head_n * a.q.head;
    const T* gp = (const T*)a.grad_out.data + row_n * a.grad_out.row + head_n * a.grad_out.head;
    int64_t stat_at = head_n * a.qs.rows + row_n;
    auto load = [&](int i) {  // tiles in turn
        if (i > 0) {
            if (xn + BQ <= i1) {
                xn += BQ;
                qp += BQ * a.q.row;
                gp += BQ * a.grad_out.row;
                stat_at += BQ;
            } else {
                const int back = xn - i0;
                xn = i0;
                qp += a.q.head - back * a.q.row;
                gp += a.grad_out.head - back * a.grad_out.row;
                stat_at += a.qs.rows - back;
            }
        }
        const int rows = i1 - xn + 1;
        FPSTOK_LDS char* buf = lds + (i & 1) * 2 * BQ * Tl::kPitch;
        dma.load(qp, off_q, a.q.row, rows, buf, wave);
        dma.load(gp, off_g, a.grad_out.row, rows, buf + BQ * Tl::kPitch, wave);
        if (wave < 2) {
            const float* src = (wave == 0 ? a.lse2 : a.delta) + stat_at;
            dma4(src, (uint32_t)(lane < rows ? lane : rows - 1) * 4u,
                 (uint32_t)(uintptr_t)(FPSTOK_LDS float*)stat[i & 1][wave]);
        }
    };
    auto arrive = [&](int i) {
        dma_wait();
        if (!tile_all.has(xn)) {
            FPSTOK_LDS char* buf = lds + (i & 1) * 2 * BQ * Tl::kPitch;
            // (a query with infinite elements has no finite score: its weights are
            // 0, or its lse and with it all it adds is not a number)
            Dma<T, DP, BQ>::finite(buf, ~0ull, tid);
            const uint32_t chunks = dma.clean(buf + BQ * Tl::kPitch, tid);
#pragma unroll 1
            for (uint32_t c = chunks; c != 0; c &= c - 1)
                bad.note(i, __builtin_ctz(c) * dma.kStep + dma.row);
        }
    };

    f32x16 dk[DB], dv[DB];
#pragma unroll
    for (int db = 0; db < DB; ++db) dk[db] = 0.0f, dv[db] = 0.0f;
    const float c = a.scale * kLog2e;
    auto block = [&](const FPSTOK_LDS char* qbuf, const float (*stat)[64], int b, int x0,
                     bool mask) {
        const FPSTOK_LDS char* gbuf = qbuf + BQ * Tl::kPitch;
        f32x16 x = 0.0f, y = 0.0f;
#pragma unroll
        for (int st = 0; st < STEPS; ++st) {
            Frag v;
            if constexpr (kVLds)
                v = Tl::row_frag(lds + kV, wave * 32 + (lane & 31), st, half);
            else
                v = vf[st];
            x = Elem<T>::mma(Tl::row_frag(qbuf, b * 32 + (lane & 31), st, half), kf[st], x);
            y = Elem<T>::mma(Tl::row_frag(gbuf, b * 32 + (lane & 31), st, half), v, y);
        }
        f32x16 w, ds;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int at = b * 32 + (e >> 2) * 8 + half * 4 + (e & 3);
            w[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[e], c, -stat[0][at]));
            ds[e] = w[e] * (y[e] - stat[1][at]);
        }
        if (mask) {
            const int at = x0 + b * 32 + half * 4 - e0;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const bool hide = (uint32_t)(at + (e >> 2) * 8 + (e & 3)) > e_span;
                w[e] = hide ? 0.0f : w[e];
                ds[e] = hide ? 0.0f : ds[e];
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const Frag fw = to_frag<T>(w, k), fs = to_frag<T>(ds, k);
#pragma unroll
            for (int db = 0; db < DB; ++db) {
                dv[db] = Elem<T>::mma(Tl::col_frag(gbuf, b * 32 + k * 16, db, lane), fw, dv[db]);
                dk[db] = Elem<T>::mma(Tl::col_frag(qbuf, b * 32 + k * 16, db, lane), fs, dk[db]);
            }
        }
    };
    bad.clear(tid);
    if (a.D < DP) dma.zero(lds, sizeof(smem), tid);
    __syncthreads();
    if (n > 0) {
        if constexpr (kVLds)
        {
            const Dma<T, DP, 128> dma_v(a.D, tid);
            dma_v.load((const T*)a.v.data + (t.k0 + t.row0) * a.v.row + t.hk * a.v.head,
                       dma_v.offset(a.v.row), a.v.row, t.rows, lds + kV, wave);
        }
        load(0);
        arrive(0);
    }
    __syncthreads();
    for (int i = 0; i < n; ++i) {
        const int x0 = xn;
        FPSTOK_LDS char* qbuf = lds + (i & 1) * 2 * BQ * Tl::kPitch;
        const float(*st)[64] = stat[i & 1];
        const float lse_here = st[0][lane];  // (on its way while the next tile is called for)
        if (i + 1 < n) load(i + 1);
        // (the bits past BQ rows are the next tile's)
        const uint64_t gone = __ballot(lse_here == INFINITY);
        if (gone != 0) {
            Dma<T, DP, BQ>::finite(qbuf, gone, tid);
            Dma<T, DP, BQ>::drop(qbuf + BQ * Tl::kPitch, gone, tid);
            if constexpr (kVLds) {
                Dma<T, DP, 128>::clean(lds + kV, tid);
            } else {
#pragma unroll
                for (int e = 0; e < STEPS; ++e) vf[e] = frag_clean<T>(vf[e]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int b = 0; b < QB; ++b)
            if (wave_live && wave_any.has(x0 + b * 32))
                block(qbuf, st, b, x0, !wave_all.has(x0 + b * 32));
        if (i + 1 < n) arrive(i + 1);
        __syncthreads();
    }
    if (a.left >= 0 && t.row0 == 0 && t.rows > 0 && wave * 32 < a.sinks && t.part == 0) {
        const int past = t.tq - 1 - last_by_window(a, t.tq, t.tk);
        const int chunks = (past + (1 << a.sink_shift) - 1) >> a.sink_shift;
        if (chunks > 0) {
            const bool mine = live && r < a.sinks;
            const int64_t first =
                a.qs.cu ? slot_of(t.q0, t.b, 1, a.sink_shift)
                        : (int64_t)t.b * ((a.qs.cap + (1 << a.sink_shift) - 1) >> a.sink_shift);
            const int64_t step = (int64_t)a.Hk * 2 * a.sinks * a.D;
            const float* part = a.sink_part + (first * a.Hk + t.hk) * 2 * a.sinks * a.D +
                                (mine ? r : 0) * a.D;
            // dK is scaled when it is stored, and so is this
            for (int x = 0; x < chunks; ++x, part += step)
#pragma unroll
                for (int db = 0; db < DB; ++db)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        using f4 = float __attribute__((ext_vector_type(4)));
                        const int d = db * 32 + g * 8 + half * 4, at = d < a.D ? d : 0;
                        const f4 pk = *(const f4*)(part + at);
                        const f4 pv = *(const f4*)(part + (int64_t)a.sinks * a.D + at);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            dk[db][g * 4 + e] += mine ? pk[e] : 0.0f;
                            dv[db][g * 4 + e] += mine ? pv[e] : 0.0f;
                        }
                    }
        }
    }
    zero_unless<DB>(dk, live);
    zero_unless<DB>(dv, live);
    // formed anew: at D = 128 no register is left to keep what follows from it
    int lane_end = lane;
    asm volatile("" : "+v"(lane_end));
    const int64_t row_end = t.k0 + t.row0 + wave * 32 + (lane_end & 31);
    // BadSum to grad_v over the queries of this workgroup's part that see this
    // key, and have weights, in tiles that the workgroup's keys do not all see
    // whole (grad_k has their delta, which is not finite either)
    auto add_hidden = [&](auto* to_v) {
        __syncthreads();
        const bool sees = live && e1 >= e0;
#pragma unroll 1
        for (int d0 = 0; d0 < a.D; d0 += 64) {
            BadSum<T> sum(d0);
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                const int g = (from + i) / per, x = i0 + (from + i - g * per) * BQ;
                if (tile_all.has(x)) continue;
                const int64_t h = (int64_t)t.hk * G + g;
#pragma unroll 1
                for (uint64_t rows = bad.of(i); rows != 0; rows &= rows - 1) {
                    const int y = x + __builtin_ctzll(rows);
                    const int64_t row = t.q0 + y;
                    if (sees && y >= e0 && y <= e1 && a.lse2[h * a.qs.rows + row] != INFINITY)
                        sum.add((const T*)a.grad_out.data + row * a.grad_out.row +
                                    h * a.grad_out.head,
                                a.D, half);
                }
            }
            if (sees) sum.store(to_v, a.D, half);
        }
    };
    if (a.k_splits > 1) {
        float* part = a.k_part + k_part_at(a, t.part, t.hk, row_end);
        float* part_v = part + k_part_at(a, 0, a.Hk, 0);
        store_row<float, DB>(dk, 1.0f, live ? part : nullptr, a.D, lane_end);
        store_row<float, DB>(dv, 1.0f, live ? part_v : nullptr, a.D, lane_end);
        if (bad.tiles != 0) add_hidden(part_v);
        return;
    }
    T* ok = (T*)a.grad_k.data + row_end * a.grad_k.row + t.hk * a.grad_k.head;
    T* ov = (T*)a.grad_v.data + row_end * a.grad_v.row + t.hk * a.grad_v.head;
    const bool write = live || r < t.pad;
    store_row<T, DB>(dk, a.scale, write ? ok : nullptr, a.D, lane_end);
    store_row<T, DB>(dv, 1.0f, write ? ov : nullptr, a.D, lane_end);
    if (bad.tiles != 0) add_hidden(ov);
}

// Adds the parts of keys whose walk was split, in order: 4 elements of one key
// and head per thread.
template <class T>
__global__ __launch_bounds__(256) void attention_join_dkv_kernel(AttnArgs a) {
    using f4 = float __attribute__((ext_vector_type(4)));
    using T4 = T __attribute__((ext_vector_type(4)));
    const uint32_t per = (uint32_t)a.D / 4;
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t at = x / per;
    const int d = (int)(x - at * per) * 4;
    const int64_t row = at / a.Hk;
    const int hk = (int)(at - row * a.Hk);
    if (row >= a.ks.rows) return;
    bool here = true;
    if (a.ks.cu) {
        if (row < cu_at(a.ks, 0) || row >= cu_at(a.ks, a.ks.B)) return;
    } else {
        here = row % a.ks.cap < a.ks.count[row / a.ks.cap];
    }
    f4 k = 0.0f, v = 0.0f;
    if (here) {
        const int64_t v_at = k_part_at(a, 0, a.Hk, 0);
#pragma unroll 4
        for (int s = 0; s < a.k_splits; ++s) {
            const float* part = a.k_part + k_part_at(a, s, hk, row) + d;
            k += *(const f4*)part;
            v += *(const f4*)(part + v_at);
        }
    }
    *(T4*)((T*)a.grad_k.data + row * a.grad_k.row + hk * a.grad_k.head + d) =
        __builtin_convertvector(k * a.scale, T4);
    *(T4*)((T*)a.grad_v.data + row * a.grad_v.row + hk * a.grad_v.head + d) =
        __builtin_convertvector(v, T4);
}

int64_t row_slots(const SeqArgs& s, int G, int shift) {
    if (s.cu) return (s.rows * G >> shift) + s.B;
    return (int64_t)s.B * (((int64_t)s.cap * G + (1 << shift) - 1) >> shift);
}

// Splits a row's keys until about `want` workgroups are there, into at least
// `least` keys each.
static int64_t key_splits(const AttnArgs& a, int64_t blocks, int64_t q_len, int64_t k_len,
                          int64_t want, int64_t least) {
    int64_t seen = k_len;
    if (a.left >= 0 && a.right >= 0 && seen > q_len + a.left + a.right + a.sinks)
        seen = q_len + a.left + a.right + a.sinks;
    int64_t n = blocks > 0 ? want / blocks : 1;
    if (n > seen / least) n = seen / least;
    return n < 1 ? 1 : n > 256 ? 256 : n;
}

AttnPlan plan_attention(const AttnArgs& a, int32_t q_len, int32_t k_len) {
    const int G = a.G;
    AttnPlan p;
    p.few = (int64_t)q_len * G <= 32;
    const int64_t blocks = row_slots(a.qs, G, p.few ? 5 : 7) * a.Hk;
    if (p.few) {
        p.splits = (int32_t)key_splits(a, blocks, q_len, k_len, 1024, 512);
    } else {
        // two workgroups per compute unit, unless nearly every one has a
        // workgroup already (5000 rows, 5 heads of 64: 200 workgroups, 2 parts
        // 74 us, unsplit 95; 2000 rows, 16 heads on 4, D = 128: 252 workgroups, 2
        // parts 59 us, unsplit 52).  How much 2 parts of 225 to 256 workgroups
        // would take goes by the keys: 1.16 times one part at 16 heads on 4 of
        // 128 and 1800 to 2050 rows, 0.97 with a causal mask; 0.95 and 0.76 at 8
        // heads of 128 and 3600 to 4100 rows; 0.77 and 0.64 at 5 heads of 64 and 5800
        // to 6500 rows, and from 257 workgroups on both are the same.  The step at
        // 224 keeps the first of these.  2500 rows of one head, parts of 256 keys
        // or more 19 us, of 512 21.  float32 tiles take 8 times as long, and four
        // workgroups even the compute units out (3000 rows, 12 heads of 64: 320
        // us, unsplit 450; 1500 rows: 114, with two 96).
        const int64_t want = a.dtype == 0 ? 1024 : blocks > 224 ? 0 : 512;
        p.splits = (int32_t)key_splits(a, blocks, 128 / G + 1, k_len, want, 256);
    }
    return p;
}

int plan_key_parts(const AttnArgs& a, int32_t q_len) {
    // workgroups of 128 keys, each with a walk of about this many queries, in at
    // most as many parts as all run at once (5000 rows, 8 heads on 1: 10 parts of
    // 40 workgroups 382 us a training step, 13 parts 430; 8 heads on 8, 320
    // workgroups: unsplit 397, 2 parts 412) and in
    // parts of 192 or more (a walk alone on its compute unit takes 1.6 us per 64
    // queries, the join 5 us.  One event of 110 tokens, 8 heads on 1, all of a
    // training step: parts of 512 or more 43 us, of 192 34; 21 padded events of
    // up to 256 tokens, 12 heads: of 192 43 us, of 128 54)
    const int64_t blocks = row_slots(a.ks, 1, 7) * a.Hk;
    int64_t walk = q_len;
    if (a.left >= 0 && a.right >= 0 && walk > 128 + a.left + a.right)
        walk = 128 + (int64_t)a.left + a.right;
    walk *= a.G;
    int64_t n = blocks > 0 ? 512 / blocks : 1;
    if (n > walk / 192) n = walk / 192;
    return n < 1 ? 1 : n > 64 ? 64 : (int)n;
}

template <class T>
static hipError_t forward(const AttnArgs& a, const AttnPlan& plan, hipStream_t s) {
    constexpr bool k16 = sizeof(T) == 2;
    const int64_t blocks = row_slots(a.qs, a.G, plan.few ? 5 : 7) * a.Hk;
    const dim3 grid((unsigned)(blocks * a.splits));
    if (plan.few) {
        if (a.D <= 64)
            attention_few_kernel<T, 64, 32><<<grid, 256, 0, s>>>(a);
        else
            attention_few_kernel<T, 128, 32><<<grid, 256, 0, s>>>(a);
    } else {
        if (a.D <= 64)
            attention_kernel<T, 64, 64><<<grid, 256, 0, s>>>(a);
        else
            attention_kernel<T, 128, k16 ? 64 : 32><<<grid, 256, 0, s>>>(a);
    }
    if (a.splits > 1) {
        // a workgroup per (query, head) for few of them (one query on 131k keys
        // in 32 parts: 175 us against 180), a thread per 4 elements for many
        // (5000 rows, 3 heads: 48 us against 64)
        const int64_t joins = (a.qs.rows * a.H * (a.D / 4) + 255) / 256;
        if (joins >= 128)
            attention_join_rows_kernel<T><<<dim3((unsigned)joins), 256, 0, s>>>(a);
        else
            attention_join_kernel<T><<<dim3((unsigned)(a.qs.rows * a.H)), 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

template <class T>
static hipError_t backward(const AttnArgs& a, hipStream_t s) {
    constexpr bool k16 = sizeof(T) == 2;
    const dim3 q((unsigned)(row_slots(a.qs, a.G, 7) * a.Hk));
    const dim3 k((unsigned)(row_slots(a.ks, 1, 7) * a.Hk * a.k_splits));
    if (a.qs.rows > 0) {
        const bool narrow = k16 && a.left >= 0 && a.right >= 0 && a.left + a.right < 32 - a.sinks;
        if (a.D <= 64) {
            if (narrow)
                attention_dq_kernel<T, 64, 64, k16><<<q, 256, 0, s>>>(a);
            else
                attention_dq_kernel<T, 64, 64, false><<<q, 256, 0, s>>>(a);
        } else {
            if (narrow)
                attention_dq_kernel<T, 128, k16 ? 64 : 32, k16><<<q, 256, 0, s>>>(a);
            else
                attention_dq_kernel<T, 128, k16 ? 64 : 32, false><<<q, 256, 0, s>>>(a);
        }
    }
    if (a.sink_part && a.qs.rows > 0) {
        const dim3 c((unsigned)(row_slots(a.qs, 1, a.sink_shift) * a.Hk));
        if (a.D <= 64)
            attention_sink_kernel<T, 64><<<c, 256, 0, s>>>(a);
        else
            attention_sink_kernel<T, 128><<<c, 256, 0, s>>>(a);
    }
    if (a.ks.rows > 0) {
        if (a.D <= 64)
            attention_dkv_kernel<T, 64, k16 ? 64 : 32><<<k, 256, 0, s>>>(a);
        else
            attention_dkv_kernel<T, 128, 32><<<k, 256, 0, s>>>(a);
        if (a.k_splits > 1) {
            const int64_t threads = a.ks.rows * a.Hk * (a.D / 4);
            attention_join_dkv_kernel<T>
                <<<dim3((unsigned)((threads + 255) / 256)), 256, 0, s>>>(a);
        }
    }
    return hipGetLastError();
}

hipError_t launch_attention(const AttnArgs& a, const AttnPlan& plan, hipStream_t s) {
    return a.dtype == 0   ? forward<float>(a, plan, s)
           : a.dtype == 1 ? forward<_Float16>(a, plan, s)
                          : forward<__bf16>(a, plan, s);
}

hipError_t launch_attention_backward(const AttnArgs& a, hipStream_t s) {
    return a.dtype == 0 ? backward<float>(a, s)
                        : a.dtype == 1 ? backward<_Float16>(a, s) : backward<__bf16>(a, s);
}

}  // namespace fpstok
