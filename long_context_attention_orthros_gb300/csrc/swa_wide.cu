// swa_wide.cu -- the base stream with attention sinks on the 5th-generation tensor cores where the window is too wide for
// swa_tc.cuh's band in tensor memory, or heads do not share K and V (rows_tc.cuh): row t sees keys j <= t with
// j > t - window or j < sinks.
//
// A piece is a tile of 128 query rows (128/G tokens x G heads of a KV head), as KEYS2, or two such tiles one behind the
// other, as ROWS2, with the key blocks of their windows and, where those begin behind block 0, that block first.  Pieces
// are shared alike by all CTAs in the order of the stream, so that a CTA's key blocks come from L2.
// ROWS2 reads and converts a key block once for 256 rows, KEYS2 is done with a tile sooner: it is taken where all tiles
// are worked on at once (1 x 2000 tokens of 8/2 heads, d = 64, window 300: 13.6 us against 18.6; 1 x 1024 of 32/8 heads,
// d = 128, window 640: 34.5 against 26.5; 1 x 8192 of 8/2 heads, d = 64, window 1024: 68 against 54; 2 x 16384 of 32/8,
// d = 128: 1151 against 852, a third of the MMAs' rate).  Bound by the chain S -> softmax -> P V.
// A row's bits depend on the form and on where its piece begins, so both are those of the whole sequence: a range of
// rows takes the form that all rows would, in pieces cut at the same tokens.  Ranges begin at multiples of 128 tokens; a
// ROWS2 piece of 256 tokens (heads that do not share K and V) that one cuts has no query in its other half.  That costs
// short ranges of long sequences time (512 rows of 1 x 8192 of 8/2 heads, d = 64, window 1024: 27.8 us, as KEYS2 18.5).
#include "rows_tc.cuh"

namespace orthros {

namespace {

template <int D, int TR>
struct WideJob {
    using Params = SwaWideParams;
    using Maps = SwaWideMaps;
    struct Where {
        long long it, it1;
    };
    struct Piece {
        int g, b, t0, t1;     // tokens t0 .. t1 - 1, of which the range has those from row_begin on
        int lo, far;          // first block of the windows; the sinks' block comes before it
        int m, plain0, plain1;
    };
    struct See {
        int lo, hi, first;  // keys lo .. hi and those below first, up to hi
    };

    static __device__ __forceinline__ void share(const Params &p, Piece &, Where &where)
    {
        if ((threadIdx.x & 31) == 0)
            where = {p.pieces * blockIdx.x / gridDim.x, p.pieces * (blockIdx.x + 1) / gridDim.x};
    }
    static __device__ __forceinline__ void next(const Params &p, const Piece &, Piece &to, Where &where)
    {
        to.m = 0;
        if (where.it >= where.it1)
            return;
        const int tok = TR / (p.Hq / p.Hkv);
        const long long stream = where.it / p.per_stream;
        to.b = static_cast<int>(stream / p.Hkv);
        to.g = static_cast<int>(stream % p.Hkv);
        to.t0 = p.row_begin / tok * tok + static_cast<int>(where.it % p.per_stream) * tok;
        to.t1 = min(p.row_end, to.t0 + tok);
        to.lo = max(0, to.t0 - p.window + 1) / 64;
        to.far = p.sinks > 0 && to.lo > 0;
        to.m = to.far + (to.t1 - 1) / 64 - to.lo + 1;
        // seen whole by every row: keys from the last row's window on, up to the first row
        to.plain0 = to.far + max(0, to.t1 - p.window + 63) / 64 - to.lo;
        to.plain1 = to.far + (to.t0 + 1) / 64 - to.lo;
        if (to.plain1 <= to.plain0)
            to.plain0 = to.plain1 = 0;
        ++where.it;
    }
    static __device__ __forceinline__ void place(const Piece &c, int &g, int &b)
    {
        g = c.g;
        b = c.b;
    }
    static __device__ __forceinline__ int row_of(const Params &, const Piece &c, int x)
    {
        return x < c.far ? 0 : (c.lo + x - c.far) * 64;
    }
    static __device__ __forceinline__ int keys(const Params &p) { return p.T; }
    static __device__ __forceinline__ const CUtensorMap *map(const Maps &m, bool v, int) { return v ? &m.v : &m.k; }
    static __device__ __forceinline__ void span(const Params &p, const Piece &c, int j0, int &end, int &lo, int &first)
    {
        end = c.t1 - j0;
        lo = max(c.t0, p.row_begin) - p.window + 1;  // what only rows before the range see may not be in place
        first = p.sinks;
    }
    static __device__ __forceinline__ const orthros_bf16 *query(const Params &p, const Piece &c, int r)
    {
        const int G = p.Hq / p.Hkv, t = c.t0 + r / G;
        if (t < p.row_begin || t >= c.t1)
            return nullptr;
        return p.q + c.b * p.q_bstride + (static_cast<long long>(t) * p.Hq + c.g * G + r % G) * D;
    }
    static __device__ __forceinline__ void vectors(const Params &p, const Piece &, const float *&alpha, const float *&beta)
    {
        alpha = p.alpha;
        beta = p.beta;
    }
    static __device__ __forceinline__ See see(const Params &p, const Piece &c, int r)
    {
        const int t = c.t0 + r / (p.Hq / p.Hkv);
        return {t < c.t1 ? t - p.window + 1 : 0x7fffffff, t < c.t1 ? t : -1, t < c.t1 ? p.sinks : 0};
    }
    static __device__ __forceinline__ unsigned long long mask(const Params &, const Piece &, const See &s, int j0)
    {
        // no difference overflows: lo > -2^31, the others and j0 lie in [-1, 2^31)
        return bits_below(s.hi - j0 + 1) & (~bits_below(s.lo < j0 ? 0 : s.lo - j0) | bits_below(s.first - j0));
    }
    static __device__ __forceinline__ RowOut out(const Params &p, const Piece &c, const See &, int r)
    {
        const int G = p.Hq / p.Hkv, t = c.t0 + r / G, h = c.g * G + r % G;
        RowOut o = {nullptr, nullptr, nullptr, nullptr, false};
        if (t >= p.row_begin && t < c.t1) {
            o.row = p.o + c.b * p.o_bstride + (static_cast<long long>(t) * p.Hq + h) * D;
            if (p.lse != nullptr)
                o.lse = p.lse + (static_cast<long long>(c.b) * p.T + t) * p.Hq + h;
        }
        return o;
    }
};

template <int D>
cudaError_t launch_t(const SwaWideMaps &maps, SwaWideParams p, cudaStream_t stream)
{
    const int G = p.Hq / p.Hkv;
    const bool two = static_cast<long long>(p.B) * p.Hkv * ((p.T + 128 / G - 1) / (128 / G)) > 152;  // tiles of all rows
    const int tok = (two ? 256 : 128) / G;
    p.per_stream = (p.row_end + tok - 1) / tok - p.row_begin / tok;
    p.pieces = static_cast<long long>(p.B) * p.Hkv * p.per_stream;
    const int ctas = static_cast<int>(p.pieces < 152 ? p.pieces : 152);
    return two ? launch_rows_tc<D, true, WideJob>(maps, p, ctas, stream)
               : launch_rows_tc<D, false, WideJob>(maps, p, ctas, stream);
}

}  // namespace

cudaError_t launch_swa_wide(int D, const SwaWideMaps &maps, const SwaWideParams &p, cudaStream_t stream)
{
    return D == 128 ? launch_t<128>(maps, p, stream) : launch_t<64>(maps, p, stream);
}

}  // namespace orthros
