// Host side of the paged-cache entry points declared in include/fp8_mqa_logits.h: argument
// checks, the choice of kernel, and the launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstdio>
#include <mutex>
#include <numeric>

#include "../../include/fp8_mqa_logits.h"
#include "cache_kernels.cuh"
#include "paged_attention_kernel.cuh"
#include "paged_host.h"
#include "paged_logits_kernel.cuh"

namespace fp8mqa {
namespace {

constexpr int kPagedMaxDevices = 64;

struct PagedDevice {
    std::mutex setting_up;
    int sm_count = 0;
    int32_t* status = nullptr;  // status word of the paged logits
    std::atomic<bool> ready{false};
};

PagedDevice g_paged[kPagedMaxDevices];
template <int kTok>
bool logits_smem()
{
    const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    return cudaFuncSetAttribute(paged_logits_kernel<kTok, true>, attr,
                                int(PagedShape<kTok, true>::kSmem)) == cudaSuccess &&
           cudaFuncSetAttribute(paged_logits_kernel<kTok, false>, attr,
                                int(PagedShape<kTok, false>::kSmem)) == cudaSuccess;
}

// CTAs of a full wave of the attention kernel.
int64_t attention_wave(int sm_count)
{
    return std::min<int64_t>(kAttnMaxCtas, int64_t(sm_count) * kAttnCtasPerSm);
}

template <int kType, int kDim, int kNT, int kHq>
bool attention_smem()
{
    return cudaFuncSetAttribute(paged_attention_kernel<kType, kDim, kNT, kHq>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                AttnShape<kType, kDim, kNT, kHq>::kSmem) == cudaSuccess;
}

template <int kType>
bool attention_smem()
{
    return attention_smem<kType, 64, 1, 1>() && attention_smem<kType, 64, 2, 1>() &&
           attention_smem<kType, 64, 2, 2>() && attention_smem<kType, 64, 2, 4>() &&
           attention_smem<kType, 128, 1, 1>() && attention_smem<kType, 128, 2, 1>() &&
           attention_smem<kType, 128, 2, 2>() && attention_smem<kType, 128, 2, 4>();
}

// Launches a kernel that begins with griddepcontrol.wait: it is set up while the one before it ends.
// Its own result says whether it is under way (the runtime's last error may be an older one of the
// caller's).
template <class... Params, class... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                  const Args&... args)
{
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int init_paged(int dev, PagedDevice& st)
{
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&st.sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return FP8MQA_ERR_CUDA;
    }
    if (major != 10 || minor != 3) return FP8MQA_ERR_ARCH;
    if (!attention_smem<FP8MQA_E4M3>() || !attention_smem<FP8MQA_BF16>() ||
        !attention_smem<FP8MQA_F16>() ||
        !logits_smem<1>() || !logits_smem<2>() || !logits_smem<4>()) {
        cudaGetLastError();
        return FP8MQA_ERR_LAUNCH;
    }
    void* buf = nullptr;
    if (cudaMalloc(&buf, 256) != cudaSuccess || cudaMemset(buf, 0, 256) != cudaSuccess) {
        cudaFree(buf);
        cudaGetLastError();
        return FP8MQA_ERR_CUDA;
    }
    st.status = static_cast<int32_t*>(buf);
    return FP8MQA_OK;
}

// The current device's state, set up by the first call that succeeds in it: what fails once (no memory
// left, a stream being captured) is tried again by the next call.
PagedDevice* paged_device(int* err)
{
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kPagedMaxDevices) {
        cudaGetLastError();
        *err = FP8MQA_ERR_CUDA;
        return nullptr;
    }
    PagedDevice& st = g_paged[dev];
    *err = FP8MQA_OK;
    if (st.ready.load(std::memory_order_acquire)) return &st;
    const std::lock_guard<std::mutex> lock(st.setting_up);
    if (!st.ready.load(std::memory_order_relaxed)) {
        *err = init_paged(dev, st);
        if (*err != FP8MQA_OK) return nullptr;
        st.ready.store(true, std::memory_order_release);
    }
    return &st;
}

bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int64_t size_of(int32_t type) { return type == FP8MQA_E4M3 ? 1 : type == FP8MQA_F32 ? 4 : 2; }

// A cache argument: sizes, type, pointers, alignment.
int check_cache(const fp8mqa_cache* c)
{
    if (!c || c->pages < 0 || c->page_size < 1 || c->heads < 1) return FP8MQA_ERR_INVALID_ARG;
    if (c->type != FP8MQA_E4M3 && c->type != FP8MQA_BF16 && c->type != FP8MQA_F16)
        return FP8MQA_ERR_INVALID_ARG;
    if ((c->dim != 64 && c->dim != 128) || c->pages > INT32_MAX / int64_t(c->page_size))
        return FP8MQA_ERR_UNSUPPORTED_SHAPE;
    if (c->pages > 0 && (!c->data || (c->type == FP8MQA_E4M3 && !c->scale)))
        return FP8MQA_ERR_INVALID_ARG;
    if ((c->type == FP8MQA_E4M3) != (c->scale != nullptr) && c->pages > 0)
        return FP8MQA_ERR_INVALID_ARG;
    // the stride of a dimension of one is never used
    const int64_t e = size_of(c->type);
    if (!on(c->data, 16) || !on(c->scale, 4) || (c->pages > 1 && c->page_stride * e % 16) ||
        (c->page_size > 1 && c->row_stride * e % 16) || (c->heads > 1 && c->head_stride * e % 16))
        return FP8MQA_ERR_MISALIGNED;
    return FP8MQA_OK;
}

// A cache as kernels see it.  One without pages has no memory; `valid` stands for it (nothing is read
// there, but copies of no bytes carry an address).
PagedView view_of(const fp8mqa_cache& c, const void* valid)
{
    const int64_t e = size_of(c.type);
    PagedView v;
    void* const none = const_cast<void*>(valid);
    v.data = static_cast<uint8_t*>(c.pages > 0 ? c.data : none);
    v.scale = c.pages > 0 ? c.scale : static_cast<float*>(none);
    v.page_stride = c.page_stride * e;
    v.row_stride = c.row_stride * e;
    v.head_stride = c.head_stride * e;
    v.scale_page_stride = c.scale_page_stride;
    v.scale_row_stride = c.scale_row_stride;
    v.scale_head_stride = c.scale_head_stride;
    v.pages = int32_t(c.pages);
    v.page_size = c.page_size;
    v.heads = c.heads;
    return v;
}

// The units that a cache's rows are counted in; false if 32 bits do not hold them.
bool row_units(const PagedView& v, RowUnits* u)
{
    // strides of dimensions of one do not count; negative ones are not taken
    const int64_t page = v.pages > 1 ? v.page_stride : 0, row = v.page_size > 1 ? v.row_stride : 0;
    const int64_t unit = std::max<int64_t>(16, std::gcd(page, row));
    if (page < 0 || row < 0 || unit > INT32_MAX ||
        (v.pages * page + v.page_size * row) / unit >= int64_t(kNoRow))
        return false;
    u->page = uint32_t(page / unit);
    u->row = uint32_t(row / unit);
    u->unit = uint32_t(unit);
    return true;
}

// What the bounds-checking build holds a launch's accesses against, from the call's arguments alone; in the
// library nothing of it is there.
#ifdef FP8MQA_DEBUG_BOUNDS
std::atomic<uint64_t> g_short[kMemKinds];  // bytes that a kind's memory is taken to be short of (tests)
#endif
void spans(PagedBounds& b, int kind, const void* from, int64_t bytes)
{
#ifdef FP8MQA_DEBUG_BOUNDS
    b.from[kind] = reinterpret_cast<uint64_t>(from);
    b.bytes[kind] = bytes > 0 ? uint64_t(bytes) - std::min(uint64_t(bytes), g_short[kind].load()) : 0;
#endif
}
PagedBounds bounds_for(const PagedDevice& st)
{
    PagedBounds b = {};
#ifdef FP8MQA_DEBUG_BOUNDS
    b.status = st.status;
#endif
    return b;
}
// Bytes from the first to past the last of n0 x n1 x n2 places, `size` bytes each, at strides in bytes.
int64_t extent(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t size)
{
    return n0 > 0 && n1 > 0 && n2 > 0 ? (n0 - 1) * s0 + (n1 - 1) * s1 + (n2 - 1) * s2 + size : 0;
}
void spans(PagedBounds& b, int which, const PagedView& c, int64_t row_bytes)
{
    spans(b, kMemData + which, c.data,
          extent(c.pages, c.page_stride, c.page_size, c.row_stride, c.heads, c.head_stride, row_bytes));
    if (c.scale)
        spans(b, kMemScale + which, c.scale,
              extent(c.pages, 4 * c.scale_page_stride, c.page_size, 4 * c.scale_row_stride, c.heads,
                     4 * c.scale_head_stride, 4));
}
void spans(PagedBounds& b, const PageTable& t, int64_t B)
{
    spans(b, kMemTable, t.ids, extent(B, 4 * t.stride, t.cols, 4, 1, 0, 4));
}

// What an entry point returns for its launches' result; a refusal is not left behind for the caller's
// next look at the last error.
int launched(cudaError_t e)
{
    if (e == cudaSuccess) return FP8MQA_OK;
    cudaGetLastError();
    return FP8MQA_ERR_LAUNCH;
}

// Rows of x that start on 16 bytes are read 16 bytes at a time, others value by value.
template <class X, int kDim, int kTensors>
cudaError_t write_tensors(const CacheWriteParams& p, cudaStream_t s)
{
    const int64_t rows = p.T * p.heads, per = kCacheThreads / (kDim / 16);
    const unsigned blocks = unsigned((rows + per - 1) / per);
    bool vec = true;
    for (int i = 0; i < kTensors; ++i)
        vec = vec && on(p.x[i], 16) && p.row_stride[i] * int64_t(sizeof(X)) % 16 == 0 &&
              p.head_stride[i] * int64_t(sizeof(X)) % 16 == 0;
    return vec ? launch_after(cache_write_kernel<X, kDim, true, kTensors>, dim3(blocks), kCacheThreads, 0, s, p)
               : launch_after(cache_write_kernel<X, kDim, false, kTensors>, dim3(blocks), kCacheThreads, 0, s, p);
}

template <class X>
cudaError_t write_rows(const CacheWriteParams& p, int32_t dim, int tensors, cudaStream_t s)
{
    if (dim == 64) return tensors == 1 ? write_tensors<X, 64, 1>(p, s) : write_tensors<X, 64, 2>(p, s);
    return tensors == 1 ? write_tensors<X, 128, 1>(p, s) : write_tensors<X, 128, 2>(p, s);
}

// A block packs about kReadTurns x kReadPieces pieces a thread (finding the rows costs a block its
// start: 66 thousand rows of 8 heads as stored take 25.3 us so and 28.6 in one turn), but no more
// than leaves two blocks an SM.
constexpr int64_t kReadTurns = 4;
template <class Out>
cudaError_t read_rows(CacheReadParams& p, int32_t dim, int sm_count, cudaStream_t s)
{
    const int64_t row_pieces = int64_t(p.cache.heads) * dim * int64_t(sizeof(Out)) / 16;
    const int64_t rows = std::min(kReadTurns * kReadPieces * kCacheThreads / row_pieces,
                                  p.total / (2 * sm_count));
    p.block_rows = int32_t(std::max<int64_t>(1, std::min<int64_t>(kReadRows, rows)));
    const unsigned blocks = unsigned((p.total + p.block_rows - 1) / p.block_rows);
    return dim == 64 ? launch_after(cache_read_kernel<Out, 64>, dim3(blocks), kCacheThreads, 0, s, p)
                     : launch_after(cache_read_kernel<Out, 128>, dim3(blocks), kCacheThreads, 0, s, p);
}

// Key heads that a CTA's warps take: two, side by side, where a CTA gets kAttnHeadTiles tiles or more
// that way (of sequences that fill the table), else one, with four steps of its positions and so fewer
// partial results.  Measured with 1, 2 and 4 (us): 64 rows of up to 20001 positions, 8 heads: 229, 218,
// 218; 16 such rows: 67, 66, 67; 8 rows: 40, 40, 44; 32 rows of up to 16385, 4 heads, 16 bits: 97 with 1,
// 94 with 2; 16 of them: 54, 53, 58; 64 rows of 2048 selected: 44.5, 43.0, 49.6.
constexpr int64_t kAttnHeadTiles = 8;

// (The lengths lie on the device, so this rule and the next take the table's width for them.  A table of
// 131072 positions over rows of up to 2048: 64 rows of 64 / 8 heads 41.0 us, 40.7 with a table of their own
// width; 16 rows of 32 / 1 heads 14.9 and 14.1; 64 rows of 64 / 1 heads 38.4 and 32.2.)
//
// The grid is a full wave, or fewer CTAs where there are fewer tiles, and a multiple of the chunks of
// heads.
template <int kType, int kDim, int kNT, int kHq>
cudaError_t attention_launch(PagedAttentionParams& p, int sm_count, cudaStream_t s)
{
    using S = AttnShape<kType, kDim, kNT, kHq>;
    const int block = kHq * S::kHeads;
    const int64_t group = p.q_heads / p.k.heads, parts = (group + block - 1) / block;
    const int64_t wave = attention_wave(sm_count);
    const int64_t longest =
        std::max<int64_t>(1, p.n_indices >= 0 ? p.n_indices : int64_t(p.table.cols) * p.k.page_size);
    p.hw = p.k.heads % 2 == 0 && kHq <= 2 ? 2 : 1;
    int64_t tile, chunks, tiles;
    for (;; p.hw = 1) {
        tile = S::kStep * (kAttnWarps / (p.hw * kHq));
        chunks = p.k.heads / p.hw * parts;
        tiles = p.B * ((longest + tile - 1) / tile);
        if (p.hw == 1 || tiles * chunks >= kAttnHeadTiles * wave) break;
    }
    const int64_t per_chunk = std::min(tiles, std::max<int64_t>(1, wave / chunks));
    const cudaError_t e = launch_after(paged_attention_kernel<kType, kDim, kNT, kHq>,
                                       dim3(unsigned(per_chunk * chunks)), kAttnThreads, S::kSmem, s, p);
    // without the first kernel there is nothing in the workspace that the second one could join
    if (e != cudaSuccess || per_chunk == 1) return e;  // per_chunk 1: nothing is split
    // of a row's blocks 32 at most have work; those of a single row come first
    const int64_t shares = p.B == 1 ? std::min<int64_t>(per_chunk - 1, 32) : per_chunk - 1;
    const dim3 grid(unsigned(shares), unsigned(chunks * p.hw * kHq * kNT));
    // a few rows of many shares want many loads for each result, many rows of a few shares many blocks:
    // one row of 456 shares takes 14.5 us in all with 8 warps a block and 16.0 with 4, 64 rows of three
    // or four 231 and 223
    if (per_chunk >= 32 * p.B)
        return launch_after(paged_attention_join_kernel<kDim, 8>, grid, 256, 0, s, p, block, int(per_chunk));
    return launch_after(paged_attention_join_kernel<kDim, 4>, grid, 128, 0, s, p, block, int(per_chunk));
}

// A warp takes up to 8 query heads of a group, or 16.  Groups of more than 16 go to two or four warps
// that share a ring where the shares are long enough (steps a warp would take if the sequences fill the
// table), else to CTAs of their own, whose warps wait for nobody.  Measured, shared and not (us): groups
// of 32 with 176 steps 458 and 492, 36 steps 84.3 and 85.8, 8 steps 58 and 51, 2 steps 23.7 and 22.9;
// groups of 64 with 22 steps 125 and 132, 9 steps 117 and 130; groups of 128 with 2 steps 73 and 67.
template <int kType, int kDim>
cudaError_t attention_heads(PagedAttentionParams& p, int sm_count, cudaStream_t s)
{
    using S = AttnShape<kType, kDim, 2, 1>;
    const int group = p.q_heads / p.k.heads;
    const int64_t longest = p.n_indices >= 0 ? p.n_indices : int64_t(p.table.cols) * p.k.page_size;
    const int64_t steps = p.B * ((longest + S::kStep - 1) / S::kStep) * p.k.heads /
                          (attention_wave(sm_count) * kAttnWarps);
    if (group <= 8) return attention_launch<kType, kDim, 1, 1>(p, sm_count, s);
    if (group <= 16 || steps < (group <= 32 ? 32 : 8)) return attention_launch<kType, kDim, 2, 1>(p, sm_count, s);
    if (group <= 32) return attention_launch<kType, kDim, 2, 2>(p, sm_count, s);
    return attention_launch<kType, kDim, 2, 4>(p, sm_count, s);
}

template <int kType>
cudaError_t attention_dim(PagedAttentionParams& p, int32_t dim, int sm_count, cudaStream_t s)
{
    return dim == 64 ? attention_heads<kType, 64>(p, sm_count, s) : attention_heads<kType, 128>(p, sm_count, s);
}

// Whether TMA fetches the keys.  It can where a page's rows lie evenly apart, pages a whole number of
// rows apart, in pieces of 8 rows or more (a piece then keeps to the swizzle's atoms), and the scales
// side by side on 16 bytes.  It pays from pieces of 32 rows on: 64 rows x 2 tokens take 33.9 us so and
// 37.3 by 16-byte copies on pages of 32, 43.3 and 40.9 on pages of 16, 30.2 and 35.9 on pages of 64.
constexpr int32_t kPagedBoxRows = 32;
bool paged_maps(PagedLogitsParams& p, uint32_t tokens, CUtensorMap* map_k, CUtensorMap* map_q)
{
    const PagedView& k = p.keys;
    const int64_t pitch = k.row_stride, step = k.pages > 1 ? k.page_stride : 0;
    if (k.pages < 1 || k.page_size % kPagedBoxRows != 0 || pitch < kPagedDim || step % pitch != 0)
        return false;
    if (k.scale_row_stride != 1 || (k.pages > 1 && k.scale_page_stride % 4 != 0) || !on(k.scale, 16))
        return false;
    const int64_t rows = (k.pages - 1) * (step / pitch) + k.page_size;
    const int64_t q_rows = p.B * p.T * kPagedHeads;
    if (rows >= int64_t(1) << 31 || q_rows >= int64_t(1) << 31) return false;
    p.box = std::min(kPagedTile, k.page_size & -k.page_size);
    p.box_shift = __builtin_ctz(unsigned(p.box));
    p.page_rows = uint32_t(step / pitch);
    return encode_rows128(map_k, k.data, uint64_t(rows), uint64_t(pitch), uint32_t(p.box)) &&
           encode_rows128(map_q, p.q, uint64_t(q_rows), kPagedDim, tokens * kPagedHeads);
}

// One launch of the paged logits, kTok tokens a CTA: a full wave, or a CTA for each tile and span.
template <int kTok>
cudaError_t logits_launch(PagedLogitsParams& p, int sm_count, cudaStream_t s)
{
    using S = PagedShape<kTok, true>;
    const int64_t work = p.B * ((p.N + kPagedTile - 1) / kPagedTile);
    const int64_t wave = int64_t(sm_count) * S::kCtasPerSm;
    const dim3 grid(unsigned(std::min(work, wave)), unsigned((p.T + kTok - 1) / kTok));
    CUtensorMap map_k = {}, map_q = {};
    if (paged_maps(p, kTok, &map_k, &map_q))
        return launch_after(paged_logits_kernel<kTok, true>, grid, S::kThreads, S::kSmem, s, p, map_k, map_q);
    return launch_after(paged_logits_kernel<kTok, false>, grid, PagedShape<kTok, false>::kThreads,
                        PagedShape<kTok, false>::kSmem, s, p, map_k, map_q);
}

}  // namespace

bool paged_take_status(int dev, int32_t* flags)
{
    const PagedDevice& st = g_paged[dev];
    if (!st.ready.load(std::memory_order_acquire)) return true;
    uint64_t word[2] = {0, 0};  // the flags, and the bounds-checking build's record
    if (cudaMemcpy(word, st.status, sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess) return false;
    if (word[1] != 0)
        std::fprintf(stderr,
                     "fp8mqa: bounds violation recorded: paged kind %u, byte offset %lld "
                     "(kinds: 1 slots, 2-3 rows, 4-5 data, 6-7 scale, 8 table, 9 lens or starts, 10 indices, "
                     "11 q, 12 w, 13 out, 14 out scale or lse, 15-16 workspace)\n",
                     unsigned(word[1] >> 48), static_cast<long long>(word[1] << 16) >> 16);
    if ((word[0] != 0 || word[1] != 0) && cudaMemset(st.status, 0, sizeof(word)) != cudaSuccess) return false;
    *flags |= int32_t(word[0]);
    return true;
}

}  // namespace fp8mqa

extern "C" {

#ifdef FP8MQA_DEBUG_BOUNDS
// For tests of the checks: a kind's memory is taken to end `bytes` earlier in the calls that follow, whose
// accesses there are then recorded and not made.
FP8MQA_API void fp8_mqa_debug_bounds_short(int32_t kind, uint64_t bytes)
{
    if (kind > 0 && kind < fp8mqa::kMemKinds) fp8mqa::g_short[kind].store(bytes);
}
#endif

int fp8_mqa_cache_write(const int32_t* slots, int64_t T, int32_t x_type, const void* x,
                        int64_t x_row_stride, int64_t x_head_stride, const fp8mqa_cache* cache,
                        const void* x2, int64_t x2_row_stride, int64_t x2_head_stride,
                        const fp8mqa_cache* cache2, void* stream)
{
    using namespace fp8mqa;
    if (T < 0 || (x2 == nullptr) != (cache2 == nullptr)) return FP8MQA_ERR_INVALID_ARG;
    if (x_type != FP8MQA_BF16 && x_type != FP8MQA_F16 && x_type != FP8MQA_F32)
        return FP8MQA_ERR_INVALID_ARG;
    int rc = check_cache(cache);
    if (rc == FP8MQA_OK && cache2) rc = check_cache(cache2);
    if (rc != FP8MQA_OK) return rc;
    if (cache->type != FP8MQA_E4M3 ||
        (cache2 && (cache2->type != FP8MQA_E4M3 || cache2->page_size != cache->page_size ||
                    cache2->heads != cache->heads || cache2->dim != cache->dim)))
        return FP8MQA_ERR_INVALID_ARG;
    if (T * cache->heads >= int64_t(1) << 31) return FP8MQA_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return FP8MQA_OK;
    if (!slots || !x) return FP8MQA_ERR_INVALID_ARG;
    const uintptr_t e = uintptr_t(size_of(x_type));
    if (!on(slots, 4) || !on(x, e) || (x2 && !on(x2, e))) return FP8MQA_ERR_MISALIGNED;
    int err = FP8MQA_OK;
    const PagedDevice* st = paged_device(&err);
    if (!st) return err;
    CacheWriteParams p;
    p.slots = slots;
    p.T = T;
    p.heads = cache->heads;
    p.by_heads = FastDiv(uint32_t(p.heads));
    p.by_page = FastDiv(uint32_t(cache->page_size));
    p.x[0] = x;
    p.x[1] = x2;
    p.row_stride[0] = x_row_stride;
    p.row_stride[1] = x2_row_stride;
    p.head_stride[0] = x_head_stride;
    p.head_stride[1] = x2_head_stride;
    p.cache[0] = view_of(*cache, x);
    p.cache[1] = view_of(cache2 ? *cache2 : *cache, x);
    p.bounds = bounds_for(*st);
    spans(p.bounds, kMemSlots, slots, 4 * T);
    for (int i = 0; i < (x2 ? 2 : 1); ++i) {
        spans(p.bounds, kMemRows + i, p.x[i],
              extent(T, p.row_stride[i] * int64_t(e), p.heads, p.head_stride[i] * int64_t(e), 1, 0, cache->dim * int64_t(e)));
        spans(p.bounds, i, p.cache[i], cache->dim);
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int tensors = x2 ? 2 : 1;
    return launched(x_type == FP8MQA_BF16  ? write_rows<__nv_bfloat16>(p, cache->dim, tensors, s)
                    : x_type == FP8MQA_F16 ? write_rows<__half>(p, cache->dim, tensors, s)
                                           : write_rows<float>(p, cache->dim, tensors, s));
}

int fp8_mqa_cache_read(const fp8mqa_cache* cache, const int32_t* table, int64_t table_stride,
                       int32_t table_cols, const int32_t* starts, int64_t B, int64_t total,
                       int32_t out_type, void* out, float* out_scale, void* stream)
{
    using namespace fp8mqa;
    const int rc = check_cache(cache);
    if (rc != FP8MQA_OK) return rc;
    if (cache->type != FP8MQA_E4M3 || B < 0 || total < 0 || table_cols < 0 || out_type < 0 ||
        out_type > FP8MQA_F32)
        return FP8MQA_ERR_INVALID_ARG;
    if (total * cache->heads >= int64_t(1) << 31 || B >= int64_t(1) << 31)
        return FP8MQA_ERR_UNSUPPORTED_SHAPE;
    if (total == 0) return FP8MQA_OK;
    if (!starts || !out || (table_cols > 0 && B > 0 && !table) ||
        (out_type == FP8MQA_E4M3) != (out_scale != nullptr))
        return FP8MQA_ERR_INVALID_ARG;
    if (!on(table, 4) || !on(starts, 4) || !on(out, 16) || !on(out_scale, 4))
        return FP8MQA_ERR_MISALIGNED;
    int err = FP8MQA_OK;
    PagedDevice* st = paged_device(&err);
    if (!st) return err;
    CacheReadParams p;
    p.cache = view_of(*cache, out);
    p.table = {table, table_stride, table_cols, FastDiv(uint32_t(cache->page_size))};
    p.starts = starts;
    p.B = B;
    p.total = total;
    p.by_heads = FastDiv(uint32_t(cache->heads));
    p.out = out;
    p.out_scale = out_scale;
    p.bounds = bounds_for(*st);
    spans(p.bounds, 0, p.cache, cache->dim);
    spans(p.bounds, p.table, B);
    spans(p.bounds, kMemLens, starts, 4 * (B + 1));
    spans(p.bounds, kMemOut, out, total * cache->heads * cache->dim * size_of(out_type));
    spans(p.bounds, kMemOutScale, out_scale, 4 * total * cache->heads);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launched(out_type == FP8MQA_E4M3   ? read_rows<uint8_t>(p, cache->dim, st->sm_count, s)
                    : out_type == FP8MQA_BF16 ? read_rows<__nv_bfloat16>(p, cache->dim, st->sm_count, s)
                    : out_type == FP8MQA_F16  ? read_rows<__half>(p, cache->dim, st->sm_count, s)
                                              : read_rows<float>(p, cache->dim, st->sm_count, s));
}

int fp8_mqa_logits_paged(const uint8_t* q_fp8, const float* w, int64_t B, int32_t T, int32_t H,
                         int32_t D, const fp8mqa_cache* keys, const int32_t* table,
                         int64_t table_stride, int32_t table_cols, const int32_t* lens, float* out,
                         int64_t ld, int64_t N, int32_t clean_logits, void* stream)
{
    using namespace fp8mqa;
    if (B < 0 || T < 0 || N < 0 || ld < N || table_cols < 0 ||
        (clean_logits != 0 && clean_logits != 1))
        return FP8MQA_ERR_INVALID_ARG;
    if (H != kPagedHeads || D != kPagedDim) return FP8MQA_ERR_UNSUPPORTED_SHAPE;
    const int rc = check_cache(keys);
    if (rc != FP8MQA_OK) return rc;
    if (keys->type != FP8MQA_E4M3 || keys->heads != 1 || keys->dim != kPagedDim)
        return FP8MQA_ERR_UNSUPPORTED_SHAPE;
    if (B * T >= int64_t(1) << 31 || T > 65535 || N >= int64_t(1) << 30) return FP8MQA_ERR_UNSUPPORTED_SHAPE;
    if (B == 0 || T == 0 || N == 0) return FP8MQA_OK;
    if (!q_fp8 || !w || !lens || !out || (table_cols > 0 && !table)) return FP8MQA_ERR_INVALID_ARG;
    if (!on(q_fp8, 16) || !on(w, 16) || !on(table, 4) || !on(lens, 4) || !on(out, 4))
        return FP8MQA_ERR_MISALIGNED;
    int err = FP8MQA_OK;
    PagedDevice* st = paged_device(&err);
    if (!st) return err;
    PagedLogitsParams p;
    p.q = q_fp8;
    p.w = w;
    p.keys = view_of(*keys, q_fp8);
    p.table = {table, table_stride, table_cols, FastDiv(uint32_t(keys->page_size))};
    p.lens = lens;
    p.out = out;
    p.ld = ld;
    p.N = N;
    p.B = B;
    p.T = T;
    p.clean = clean_logits;
    p.status = st->status;
    p.wait_ns = wait_limit_ns();
    p.suspend_ns = uint32_t(std::clamp<uint64_t>(p.wait_ns, 32, kPagedSuspendNs));
    if (!row_units(p.keys, &p.units)) return FP8MQA_ERR_UNSUPPORTED_SHAPE;
    p.bounds = bounds_for(*st);
    spans(p.bounds, 0, p.keys, kPagedDim);
    spans(p.bounds, p.table, B);
    spans(p.bounds, kMemLens, lens, 4 * B);
    spans(p.bounds, kMemQ, q_fp8, B * T * kPagedHeads * kPagedDim);
    spans(p.bounds, kMemW, w, B * T * kPagedHeads * 4);
    spans(p.bounds, kMemOut, out, extent(B * T, 4 * ld, N, 4, 1, 0, 4));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launched(T == 1   ? logits_launch<1>(p, st->sm_count, s)
                    : T == 2 ? logits_launch<2>(p, st->sm_count, s)
                             : logits_launch<4>(p, st->sm_count, s));
}

uint64_t fp8_mqa_attention_paged_workspace_bytes(int32_t q_heads, int32_t kv_heads, int32_t dim)
{
    using namespace fp8mqa;
    int err = FP8MQA_OK;
    if (q_heads < 1 || kv_heads < 1 || dim < 1) return 0;
    const PagedDevice* st = paged_device(&err);
    if (!st) return 0;
    // two partial results a CTA (heads x dim sums, and each head's m and l); a launch with more
    // chunks of heads than a wave has CTAs splits no row
    const int32_t group = q_heads / kv_heads;
    const uint64_t heads =
        group > 32 ? 64 : (group > 16 ? 32 : group > 8 ? 16 : 8) * (kv_heads % 2 == 0 ? 2 : 1);
    return kAttnMaxCtas * sizeof(AttnSplit) +
           2 * uint64_t(attention_wave(st->sm_count)) * heads * uint64_t(dim + 2) * sizeof(float);
}

int fp8_mqa_attention_paged(const void* q, int32_t q_type, int64_t B, int32_t q_heads,
                            int64_t q_row_stride, int64_t q_head_stride, const fp8mqa_cache* k,
                            const fp8mqa_cache* v, const int32_t* table, int64_t table_stride,
                            int32_t table_cols, const int32_t* lens, const int32_t* indices,
                            int64_t indices_stride, int32_t n_indices, float sm_scale, void* out,
                            float* lse, void* workspace, uint64_t workspace_bytes, void* stream)
{
    using namespace fp8mqa;
    if (B < 0 || q_heads < 1 || table_cols < 0 || n_indices < -1 ||
        (q_type != FP8MQA_BF16 && q_type != FP8MQA_F16))
        return FP8MQA_ERR_INVALID_ARG;
    int rc = check_cache(k);
    if (rc == FP8MQA_OK) rc = check_cache(v);
    if (rc != FP8MQA_OK) return rc;
    if (k->type != v->type || k->page_size != v->page_size || k->heads != v->heads ||
        k->dim != v->dim || q_heads % k->heads != 0 ||
        (k->type != FP8MQA_E4M3 && k->type != q_type))
        return FP8MQA_ERR_INVALID_ARG;
    // tiles (of 16 positions or more) are counted in 32 bits, and so are positions, up to a few steps
    // (of 128 positions at most) past a row's end
    const int64_t longest = n_indices >= 0 ? n_indices : int64_t(table_cols) * k->page_size;
    if (B >= int64_t(1) << 31 || longest > kAttnMaxPositions || B * (longest / 16 + 1) >= int64_t(1) << 31)
        return FP8MQA_ERR_UNSUPPORTED_SHAPE;
    if (B == 0) return FP8MQA_OK;
    if (!q || !lens || !out || !workspace || (table_cols > 0 && !table) ||
        (n_indices > 0 && !indices))
        return FP8MQA_ERR_INVALID_ARG;
    if (!on(q, 16) || (B > 1 && q_row_stride % 8) || (q_heads > 1 && q_head_stride % 8) || !on(out, 16) || !on(lens, 4) ||
        !on(table, 4) || !on(indices, 4) || !on(lse, 4) || !on(workspace, 256))
        return FP8MQA_ERR_MISALIGNED;
    int err = FP8MQA_OK;
    PagedDevice* st = paged_device(&err);
    if (!st) return err;
    if (workspace_bytes < fp8_mqa_attention_paged_workspace_bytes(q_heads, k->heads, k->dim))
        return FP8MQA_ERR_INVALID_ARG;
    PagedAttentionParams p;
    p.q = q;
    p.q_row_stride = q_row_stride;
    p.q_head_stride = q_head_stride;
    p.k = view_of(*k, q);
    p.v = view_of(*v, q);
    p.k.pages = p.v.pages = p.k.pages < p.v.pages ? p.k.pages : p.v.pages;
    if (!row_units(p.k, &p.k_units) || !row_units(p.v, &p.v_units))
        return FP8MQA_ERR_UNSUPPORTED_SHAPE;
    p.same_rows = p.k_units.page == p.v_units.page && p.k_units.row == p.v_units.row;
    p.table = {table, table_stride, table_cols, FastDiv(uint32_t(k->page_size))};
    p.lens = lens;
    p.indices = indices;
    p.indices_stride = indices_stride;
    p.n_indices = n_indices;
    p.q_heads = q_heads;
    p.B = B;
    p.sm_scale = sm_scale;
    p.out = out;
    p.lse = lse;
    p.q_bf16 = q_type == FP8MQA_BF16;
    p.splits = static_cast<AttnSplit*>(workspace);
    p.partial = reinterpret_cast<float*>(p.splits + kAttnMaxCtas);
    p.bounds = bounds_for(*st);
    spans(p.bounds, 0, p.k, k->dim * size_of(k->type));
    spans(p.bounds, 1, p.v, v->dim * size_of(v->type));
    spans(p.bounds, p.table, B);
    spans(p.bounds, kMemLens, lens, 4 * B);
    spans(p.bounds, kMemIndices, indices, extent(B, 4 * indices_stride, n_indices, 4, 1, 0, 4));
    spans(p.bounds, kMemQ, q, extent(B, 2 * q_row_stride, q_heads, 2 * q_head_stride, 1, 0, 2 * int64_t(k->dim)));
    spans(p.bounds, kMemOut, out, B * q_heads * k->dim * 2);
    spans(p.bounds, kMemOutScale, lse, lse ? 4 * B * q_heads : 0);
    spans(p.bounds, kMemSplits, p.splits, kAttnMaxCtas * int64_t(sizeof(AttnSplit)));
    spans(p.bounds, kMemPartial, p.partial, int64_t(workspace_bytes - kAttnMaxCtas * sizeof(AttnSplit)));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launched(k->type == FP8MQA_E4M3   ? attention_dim<FP8MQA_E4M3>(p, k->dim, st->sm_count, s)
                    : k->type == FP8MQA_BF16 ? attention_dim<FP8MQA_BF16>(p, k->dim, st->sm_count, s)
                                             : attention_dim<FP8MQA_F16>(p, k->dim, st->sm_count, s));
}

}  // extern "C"
