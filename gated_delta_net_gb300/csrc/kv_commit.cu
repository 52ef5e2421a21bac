// kv_commit.cu -- an accepted path's keys and values to the slots of committed tokens, in place.
//
// Entry i of a path that ascends moves from slot len + path[i] to len + i, and path[i] >= i: taken in order, no slot is
// written before it has been read.  A block takes one head's keys or values of a request, reads the rows of
// kPieces x kThreads pieces into registers and writes them after a barrier.  Bound by memory, and for few tokens by the
// launch and its chain of loads: 64 paths of 26 to 51 nodes, 8 heads of 128, 12 us in a loop of calls, as one path takes 15 (the
// host's).
#include "attn.cuh"

namespace gdn {
namespace {

using attn::launch_dependent;

constexpr int kThreads = 128, kPieces = 4, kLongest = 1 << 20;  // entries of a path, so that its pieces can be counted in 32 bits

struct CommitParams {
    int hkv, page_size, n_pages, max_pages, row_bits, total_path;
    int64_t page_stride, slot_stride, head_stride;  // in pieces
    void *k, *v;
    const int32_t *table, *lens, *node_offsets, *path_offsets, *path;
    int32_t *new_lens, *status;
};

template <typename P>
__global__ void __launch_bounds__(kThreads) commit_kernel(CommitParams p) {
    after_previous();
    const int b = blockIdx.x / p.hkv, h = blockIdx.x % p.hkv, tid = threadIdx.x;
    const int len = p.lens[b];
    const int lo = p.path_offsets[b], hi = p.path_offsets[b + 1], n_lo = p.node_offsets[b], n_hi = p.node_offsets[b + 1];
    int bad = 0;
    if (lo < 0 || hi < lo || hi > p.total_path || n_lo < 0 || n_hi < n_lo) bad = GDN_DEV_BAD_DESC;
    if (!bad && hi - lo > kLongest) bad = GDN_DEV_BAD_PATH;
    const int n = bad || len == -1 ? 0 : hi - lo;
    if (!bad && len < -1) bad = GDN_DEV_BAD_PAGE;
    const int32_t *table = p.table + (int64_t)b * p.max_pages;
    if (!bad) {
        int wrong = 0;
        for (int i = tid; i < n; i += kThreads) {
            const int at = p.path[lo + i];
            if (at >= n_hi - n_lo || at < 0 || (i > 0 && p.path[lo + i - 1] >= at)) {
                wrong |= GDN_DEV_BAD_PATH;
                continue;
            }
            // (a table has at most 2^30 slots)
            const int64_t slot = (int64_t)len + at;
            const int from = slot < 1 << 30 ? (int)slot / p.page_size : p.max_pages;
            const int to = from < p.max_pages ? (len + i) / p.page_size : 0;  // past the table where the path does not ascend
            if (from >= p.max_pages || to >= p.max_pages || table[from] < 0 || table[from] >= p.n_pages || table[to] < 0 || table[to] >= p.n_pages)
                wrong |= GDN_DEV_BAD_PAGE;
        }
        if (__syncthreads_or(wrong & GDN_DEV_BAD_PATH)) bad |= GDN_DEV_BAD_PATH;
        if (__syncthreads_or(wrong & GDN_DEV_BAD_PAGE)) bad |= GDN_DEV_BAD_PAGE;
    }
    if (h == 0 && blockIdx.y == 0 && tid == 0) {
        if (bad) flag(p.status, bad);
        if (p.new_lens) p.new_lens[b] = bad ? len : len + n;
    }
    if (bad) return;
    P *pool = static_cast<P *>(blockIdx.y ? p.v : p.k) + h * p.head_stride;
    const int pieces = n << p.row_bits;
    for (int first = 0; first < pieces; first += kPieces * kThreads) {
        P x[kPieces];
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const int at = first + j * kThreads + tid;
            if (at < pieces) {
                const int slot = len + p.path[lo + (at >> p.row_bits)], page = slot / p.page_size;
                x[j] = pool[table[page] * p.page_stride + (slot - page * p.page_size) * p.slot_stride + (at & ((1 << p.row_bits) - 1))];
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const int at = first + j * kThreads + tid;
            if (at < pieces) {
                const int slot = len + (at >> p.row_bits), page = slot / p.page_size;
                pool[table[page] * p.page_stride + (slot - page * p.page_size) * p.slot_stride + (at & ((1 << p.row_bits) - 1))] = x[j];
            }
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_kv_commit(const gdn_kv_commit_args &a, cudaStream_t stream) {
    const gdn_kv_cache &c = a.cache;
    const int e = c.dtype == GDN_BF16 ? 2 : 4;
    CommitParams p = {};
    const bool vec = ((reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v)) & 15) == 0 &&
                     (c.page_stride | c.slot_stride | c.head_stride) * e % 16 == 0;
    const int piece = vec ? 16 / e : 1;  // entries
    p.hkv = c.n_kv_heads; p.page_size = c.page_size; p.n_pages = c.n_pages; p.max_pages = c.max_pages;
    p.row_bits = __builtin_ctz((unsigned)(c.d / piece)); p.total_path = a.total_path;
    p.page_stride = c.page_stride / piece; p.slot_stride = c.slot_stride / piece; p.head_stride = c.head_stride / piece;
    p.k = c.k; p.v = c.v; p.table = c.page_table; p.lens = c.lens;
    p.node_offsets = a.node_offsets; p.path_offsets = a.path_offsets; p.path = a.path_idx;
    p.new_lens = a.new_lens; p.status = c.dev_status;
    auto kernel = vec ? commit_kernel<uint4> : e == 2 ? commit_kernel<uint16_t> : commit_kernel<uint32_t>;
    return launch_dependent(kernel, dim3((unsigned)(c.batch * c.n_kv_heads), 2), kThreads, 0, stream, p);
}

}  // namespace gdn
