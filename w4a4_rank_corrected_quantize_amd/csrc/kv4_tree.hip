// kv4_tree.hip -- drafted tokens as a tree: their mask, places and slots from
// the nodes' parents, and the move of an accepted path to where the next
// tokens follow it.  Both are a few bytes per token and bound by latency: one
// launch each, no length known to the host.  Measured: the plan of 8 nodes 2.6
// us, of 16 x 24 .. 64 nodes 5.1, of 9 x 1 .. 130 nodes 4.7 (a walk per row up to the
// root 7.4); a path of 8 nodes, 8 heads of 128, 2.9 us; 64 paths of up to 64 nodes, 8
// heads, 7.0 us (a node at a time 10.6).
#include "kv4.h"

namespace svdq {
namespace {

__device__ __forceinline__ int kt_clamp(int x, int lo, int hi) { return min(max(x, lo), hi); }

// A slot of place `at` of a sequence, -1 for a place or page that is none.
__device__ __forceinline__ int kt_slot(const Kv4Tables &s, int seq, int64_t at)
{
    if (at < 0 || at >= (int64_t)s.width << s.page_shift) return -1;
    const int page = s.table[(int64_t)seq * s.width + (at >> s.page_shift)];
    return (uint32_t)page < (uint32_t)s.pages ? (page << s.page_shift) + (int)(at & ((1 << s.page_shift) - 1)) : -1;
}

// Up to 256 rows: a thread per row, whose mask and nearest unmet ancestor double
// their reach in every round, mask_i |= mask_a, a = ancestor of a; the depth is the
// number of bits.  More rows: a thread walks from its node up to the root.  Parents
// come before their children, so both end, and the walk meets the mask's words from
// the last to the first.
constexpr int KT_LDS = 2048, KT_FAST = 256;

__global__ __launch_bounds__(256) void kv4_tree_plan_kernel(const int32_t *__restrict__ parent, Kv4Tables s, int T, int B,
                                                            uint32_t *__restrict__ mask, int words,
                                                            int32_t *__restrict__ position,
                                                            int32_t *__restrict__ slots)
{
    __shared__ int up[KT_LDS];
    __shared__ uint32_t seen[2][KT_FAST / 32 * KT_FAST];
    const int seq = blockIdx.x, tid = threadIdx.x;
    // rows of no sequence have no slot: appended with the others they write nothing
    auto none = [&](int from, int to) {
        if (slots)
            for (int i = from + tid; i < to; i += 256) slots[i] = -1;
    };
    if (B == 0) return none(0, T);
    const int q0 = kt_clamp(s.q_start[seq], 0, T), n = kt_clamp(s.q_start[seq + 1], q0, T) - q0;
    const int kv = kt_clamp(s.kv_len[seq], 0, s.width << s.page_shift);
    if (seq == 0) none(0, q0);
    if (seq == B - 1) none(q0 + n, T);
    if (n <= KT_FAST) {
        const int own = (n + 31) >> 5;                     // words that hold bits
        const bool in = tid < n;
        int a = in ? parent[q0 + tid] : -1;
        a = a >= 0 && a < tid ? a : -1;                    // a parent that is none: a root
        const int slot = in && slots ? kt_slot(s, seq, (int64_t)kv - n + tid) : 0;
        uint32_t m[KT_FAST / 32];
#pragma unroll
        for (int w = 0; w < KT_FAST / 32; ++w) m[w] = w == tid >> 5 ? 1u << (tid & 31) : 0u;
        // after r rounds a row has met 2^r - 1 ancestors, of at most n - 1
        for (int r = 0; 1 << r < n; ++r) {
            int *ups = up + (r & 1) * KT_FAST;
            uint32_t *sees = seen[r & 1] + tid;
            if (in) {
                ups[tid] = a;
#pragma unroll
                for (int w = 0; w < KT_FAST / 32; ++w)
                    if (w < own) sees[w * KT_FAST] = m[w];
            }
            __syncthreads();                               // the round before the last has been read
            if (a >= 0) {
#pragma unroll
                for (int w = 0; w < KT_FAST / 32; ++w)
                    if (w < own) m[w] |= sees[w * KT_FAST + a - tid];
                a = ups[a];
            }
        }
        if (!in) return;
        uint32_t *row = mask + (int64_t)(q0 + tid) * words;
        int bits = 0;
#pragma unroll
        for (int w = 0; w < KT_FAST / 32; ++w) {
            bits += __popc(m[w]);
            if (w < words) row[w] = m[w];
        }
        for (int w = KT_FAST / 32; w < words; ++w) row[w] = 0;
        if (position) position[q0 + tid] = kv - n + bits - 1;
        if (slots) slots[q0 + tid] = slot;
        return;
    }
    for (int i = tid; i < min(n, KT_LDS); i += 256) up[i] = parent[q0 + i];
    __syncthreads();
    for (int i = tid; i < n; i += 256) {
        uint32_t *row = mask + (int64_t)(q0 + i) * words;
        int w = words - 1, depth = -1;
        uint32_t bits = 0;
        for (int j = i; j >= 0;) {
            for (; w > j >> 5; --w) row[w] = bits, bits = 0;
            if (w == j >> 5) bits |= 1u << (j & 31);
            ++depth;
            const int p = j < KT_LDS ? up[j] : parent[q0 + j];
            j = p < j ? p : -1;                            // a parent that is none: a root
        }
        for (; w >= 0; --w) row[w] = bits, bits = 0;
        if (position) position[q0 + i] = kv - n + depth;
        if (slots) slots[q0 + i] = kt_slot(s, seq, (int64_t)kv - n + i);
    }
}

// Pieces of one token and head: the dwords of K's codes, the codes of V that lie in
// one lane's part (a byte in every dword of D / 8 bytes), the scales.
template <bool INT4, int D>
struct KtToken {
    static constexpr int NG = INT4 ? D / 64 : D / 32, KD = D / 8, VB = D / 32;
    static constexpr int kUnits = KD + 16 + 2 * NG;
};

// A block moves one sequence's path in one head.  It reads the pieces of 64
// tokens, waits for all of them, and writes: a path's nodes ascend, so a node
// lies at or behind its new place, and nothing that is written is read later.
template <bool INT4, int D>
__global__ __launch_bounds__(256) void kv4_keep_path_kernel(Kv4View c, Kv4Tables s, int T,
                                                            const int32_t *__restrict__ path, int max_path,
                                                            int32_t *__restrict__ new_len)
{
    typedef KtToken<INT4, D> Tok;
    constexpr int NG = Tok::NG, CHUNK = 64;
    __shared__ int src[CHUNK], dst[CHUNK], found;
    const int head = blockIdx.x % c.heads, seq = blockIdx.x / c.heads, tid = threadIdx.x;
    const int32_t *nodes = path + (int64_t)seq * max_path;
    int next = tid < min(CHUNK, max_path) ? nodes[tid] : -1;        // beside the lengths, which it does not wait for
    const int q0 = kt_clamp(s.q_start[seq], 0, T), n = kt_clamp(s.q_start[seq + 1], q0, T) - q0;
    const int kv = kt_clamp(s.kv_len[seq], 0, s.width << s.page_shift);
    const int most = min(max_path, n);
    int kept = 0;
    bool more = true;
    for (int at = 0; at < most && more; at += CHUNK) {
        // the chunk's nodes: a path ends at the first that is not behind the one before it
        const int left = min(CHUNK, most - at);
        __syncthreads();
        if (tid < CHUNK) {
            const int i = at + tid, node = next;
            int before = __shfl_up(node, 1);
            if (tid == 0) before = at > 0 ? nodes[at - 1] : -1;
            next = i + CHUNK < max_path ? nodes[i + CHUNK] : -1;
            const uint64_t bad = ~__ballot(tid < left && node > before && node < n);
            const int count = bad ? __builtin_ctzll(bad) : CHUNK;
            const int64_t base = (int64_t)kv - n;
            const bool move = tid < count && node != i;
            const int a = move ? kt_slot(s, seq, base + node) : -1, b = move ? kt_slot(s, seq, base + i) : -1;
            src[tid] = b >= 0 ? a : -1, dst[tid] = b;
            if (tid == 0) found = count;
        }
        __syncthreads();
        const int count = found;
        kept += count;
        more = count == CHUNK;
        constexpr int UNITS = Tok::kUnits, PER = (CHUNK * UNITS + 255) / 256;
        uint32_t held[PER];
        // unit u of the token in `slot`: its place, and which of the three it is
        auto place = [&](int slot, int u, uint8_t *&p) {
            const size_t page = (size_t)(slot >> c.page_shift);
            const int in = slot & ((1 << c.page_shift) - 1), r = in & 15;
            const size_t run = (((page * c.heads + head) << c.page_shift) + in) >> 4;
            if (u < Tok::KD) {
                p = c.k_codes + run * (8 * D) + kv4_k_offset<INT4>(r, 8 * u, D);
                return 0;
            }
            u -= Tok::KD;
            if (u < 16) {
                p = c.v_codes + run * (8 * D) + kv4_v_offset(r, 0, u, D);
                return 1;
            }
            u -= 16;
            void *sc = u < NG ? c.k_scales : c.v_scales;
            u = u < NG ? u : u - NG;
            p = (uint8_t *)sc + (run * (16 * NG) + 16 * u + r) * (INT4 ? 4 : 1);
            return 2;
        };
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            if (256 * k >= count * UNITS) break;
            const int e = tid + 256 * k, tok = e / UNITS, u = e % UNITS;
            held[k] = 0;
            if (tok >= count || src[tok] < 0) continue;
            uint8_t *p;
            const int kind = place(src[tok], u, p);
            if (kind == 1) {
#pragma unroll
                for (int i = 0; i < Tok::VB; ++i) held[k] |= (uint32_t)p[4 * i] << (8 * i);
            } else if (INT4 || kind == 0) {
                held[k] = *reinterpret_cast<const uint32_t *>(p);
            } else {
                held[k] = *p;
            }
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wave's pieces have arrived
        __syncthreads();                                   // and every wave's
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            if (256 * k >= count * UNITS) break;
            const int e = tid + 256 * k, tok = e / UNITS, u = e % UNITS;
            if (tok >= count || src[tok] < 0) continue;
            uint8_t *p;
            const int kind = place(dst[tok], u, p);
            if (kind == 1) {
#pragma unroll
                for (int i = 0; i < Tok::VB; ++i) p[4 * i] = (uint8_t)(held[k] >> (8 * i));
            } else if (INT4 || kind == 0) {
                *reinterpret_cast<uint32_t *>(p) = held[k];
            } else {
                *p = (uint8_t)held[k];
            }
        }
    }
    if (head == 0 && tid == 0) new_len[seq] = kv - n + kept;
}

}  // namespace

hipError_t launch_kv4_tree_plan(const int32_t *parent, const Kv4Tables &s, int B, int T, uint32_t *mask, int words,
                                int32_t *position, int32_t *slots, hipStream_t stream)
{
    kv4_tree_plan_kernel<<<B > 0 ? B : 1, 256, 0, stream>>>(parent, s, T, B, mask, words, position, slots);
    return hipGetLastError();
}

hipError_t launch_kv4_keep_path(const Kv4View &c, const Kv4Tables &s, int B, int T, const int32_t *path, int max_path,
                                int32_t *new_len, hipStream_t stream)
{
    const uint32_t grid = (uint32_t)B * c.heads;
    if (c.int4 && c.dim == 64) kv4_keep_path_kernel<true, 64><<<grid, 256, 0, stream>>>(c, s, T, path, max_path, new_len);
    else if (c.int4) kv4_keep_path_kernel<true, 128><<<grid, 256, 0, stream>>>(c, s, T, path, max_path, new_len);
    else if (c.dim == 64) kv4_keep_path_kernel<false, 64><<<grid, 256, 0, stream>>>(c, s, T, path, max_path, new_len);
    else kv4_keep_path_kernel<false, 128><<<grid, 256, 0, stream>>>(c, s, T, path, max_path, new_len);
    return hipGetLastError();
}

}  // namespace svdq
