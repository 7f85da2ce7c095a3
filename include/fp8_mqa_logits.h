/*
 * fp8_mqa_logits.h -- C ABI of the GB300 (sm_103a) prefill FP8 MQA indexer-logits library.
 *
 * The operation (ROCm/aiter PR #7183 "[HIP] [JIT] Add gfx950 prefill FP8 MQA logits",
 * section "Motivation", the displayed formula):
 *
 *     out[m, n] = kv_scale[n] * sum_{h < H} relu( Q[m,h,:] . K[n,:] ) * w[m,h]
 *                 for n in [ks[m], ke[m]),   -inf elsewhere (clean_logits = 1).
 *
 * Operator contract (same page, "PR-specific question" and "Motivation"): H = 32 heads,
 * D = 128 head dimension, FP8 Q/K, float32 kv_scale / w / out, int32 row bounds, all
 * contiguous row-major.  FP8 here means OCP E4M3 ("e4m3fn", largest finite value 448).
 *
 * Conventions shared by every entry point below:
 *   - All tensor pointers are DEVICE pointers (cudaMalloc / torch CUDA memory) owned by
 *     the caller, unless an entry point says otherwise.  The library never frees them.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Compute entry
 *     points are asynchronous and stream-ordered: they return after enqueueing work.
 *   - Return value: FP8MQA_OK (0) or a negative fp8mqa_status.  Argument errors are
 *     detected on the host BEFORE anything is enqueued; the library never aborts or
 *     exits the process and throws no exceptions.
 *   - The library keeps one small device buffer per device (about 260 KB: scheduler
 *     slots and a status word), allocated on the first compute call on that device and
 *     kept until process exit.  That first call therefore must not be made while the
 *     stream is being captured into a CUDA graph.
 *   - Scheduler slots.  Each launch's work queue lives in a slot of that buffer.  Direct
 *     launches take slots from a ring of 256 in turn, so more than 256 launches running
 *     at the same moment (on many streams) would share slots and produce wrong output.
 *     A launch made while its stream is being captured into a CUDA graph gets a slot of
 *     its own that no other launch ever uses (a graph's kernel keeps its slot for every
 *     replay); up to 16384 launches can be captured per device and process, after which
 *     capturing returns FP8MQA_ERR_CAPACITY.  Replays of one instantiated graph are
 *     ordered by CUDA; two instantiations of the same captured graph must not run at
 *     the same time.
 */
#ifndef FP8_MQA_LOGITS_H
#define FP8_MQA_LOGITS_H

#include <stdint.h>

#if defined(__GNUC__)
#define FP8MQA_API __attribute__((visibility("default")))
#else
#define FP8MQA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
enum fp8mqa_status {
    FP8MQA_OK = 0,
    FP8MQA_ERR_INVALID_ARG = -1,       /* null pointer, negative size, bad flag, bad split_n */
    FP8MQA_ERR_UNSUPPORTED_SHAPE = -2, /* H != 32, D != 128, or a size beyond the limits   */
    FP8MQA_ERR_MISALIGNED = -3,        /* q/k/w/kv_scale not 16-byte aligned, out/ks/ke not 4 */
    FP8MQA_ERR_ARCH = -4,              /* current device is not compute capability 10.3     */
    FP8MQA_ERR_LAUNCH = -5,            /* the kernel could not be configured or launched    */
    FP8MQA_ERR_TIMEOUT = -6,           /* a bounded on-device wait gave up (see check_error) */
    FP8MQA_ERR_CUDA = -7,              /* a CUDA runtime call failed                        */
    FP8MQA_ERR_BOUNDS = -8,            /* a bounds-checking build found a bad access        */
    FP8MQA_ERR_CAPACITY = -9           /* no scheduler slot left for another captured launch */
};

/*
 * fp8_mqa_logits -- the logits of every query row against its key window.
 *
 *   q_fp8     [M, H, D] E4M3 bytes, row-major (query row m, head h, dim d at
 *             (m*H + h)*D + d).  16-byte aligned.
 *   k_fp8     [N, D] E4M3 bytes, row-major.  16-byte aligned.
 *   kv_scale  [N] float32, per-key scale, applied after the head sum.  16-byte aligned.
 *   w         [M, H] float32, per-(row, head) weight, applied after relu.  16-byte aligned.
 *   ks, ke    [M] int32: row m attends keys n with ks[m] <= n < ke[m].  Bounds are
 *             clamped to [0, N); ks[m] >= ke[m] is an empty row.  4-byte aligned.
 *   out       [M, N] float32, row-major, 4-byte aligned.  In-window entries are always
 *             written.  clean_logits = 1: every out-of-window entry is written with -inf
 *             (IEEE 0xff800000), so the whole matrix is defined.  clean_logits = 0:
 *             out-of-window entries are not written at all (they keep whatever the
 *             caller put there; "caller-managed output masks", page section
 *             "PR Self-Review / Behavior and intent").
 *   M, N      query rows and keys (>= 0).  M = 0 or N = 0 enqueues nothing and returns OK.
 *             Limits: M*H < 2^31, N < 2^31.
 *   H, D      must be 32 and 128 (FP8MQA_ERR_UNSUPPORTED_SHAPE otherwise).
 *   split_n   0 = automatic; > 0 = split each row block's key range into that many
 *             chunks scheduled independently (the page's "SplitN", section "Design /
 *             Grid choice" and "Known limitations").  Values above ceil(N/128) are
 *             clamped.  The result is bit-identical for every split_n.
 *   stream    cudaStream_t to enqueue on.
 *
 * Numerics: the dot products are exact (FP8 products accumulate in fp32 on the tensor
 * cores); relu, the w-weighted head sum and the kv_scale multiply are fp32.
 * Asynchronous device-side failures (a bounded wait that gave up) are reported by
 * fp8_mqa_logits_check_error.
 */
FP8MQA_API int fp8_mqa_logits(const uint8_t* q_fp8, const uint8_t* k_fp8, const float* kv_scale,
                   const float* w, const int32_t* ks, const int32_t* ke, float* out,
                   int64_t M, int64_t N, int32_t H, int32_t D, int32_t clean_logits,
                   int32_t split_n, void* stream);

/*
 * fp8_mqa_logits_is_supported -- 1 if (M, N, H, D) is inside this library's contract
 * (H = 32, D = 128, M >= 0, N >= 0, M*H < 2^31, N < 2^31) and, for device >= 0, CUDA
 * device `device` exists and has compute capability 10.3; else 0 (the page's
 * is_supported(), section "Motivation").  With device < 0 it is pure host arithmetic and
 * may be called without a GPU; with device >= 0 it only queries device attributes (it
 * launches and allocates nothing).
 */
FP8MQA_API int fp8_mqa_logits_is_supported(int64_t M, int64_t N, int32_t H, int32_t D,
                                           int32_t device);

/*
 * fp8_mqa_logits_default_split -- the split_n that split_n = 0 selects for an
 * (M, N) problem on a GPU with `num_sms` multiprocessors.  Host arithmetic only.
 */
FP8MQA_API int fp8_mqa_logits_default_split(int64_t M, int64_t N, int32_t num_sms);

/*
 * fp8_mqa_logits_check_error -- synchronizes `stream`, then reads and clears the
 * current device's status words: the one of fp8_mqa_logits / fp8_mqa_logits_host and the
 * one of fp8_mqa_logits_noalloc (each only if a call has set it up; this call allocates
 * nothing).  Returns FP8MQA_ERR_TIMEOUT if a launch since the last check had a bounded
 * on-device wait give up (its output is then incomplete), FP8MQA_ERR_BOUNDS if a
 * bounds-checking build of the library recorded an out-of-range access,
 * FP8MQA_ERR_CUDA if the synchronization or a read failed, else FP8MQA_OK.
 */
FP8MQA_API int fp8_mqa_logits_check_error(void* stream);

/*
 * fp8_mqa_logits_set_wait_limit_ns -- sets how long one on-device pipeline wait may last
 * before the kernel gives up (FP8MQA_ERR_TIMEOUT, reported by check_error), for launches
 * enqueued after the call; 0 restores the default of 1 s.  Returns the previous limit.
 * A kernel that gives up still waits for its own copies and tensor-core work in flight
 * (for up to 1 s more) before it frees its resources and exits; the next launch is
 * unaffected.  Meant for diagnostics and for testing that failure path; a limit far
 * below a call's duration makes every call fail.  Host only; process-wide.
 */
FP8MQA_API uint64_t fp8_mqa_logits_set_wait_limit_ns(uint64_t ns);

/*
 * fp8_mqa_logits_host_workspace_bytes -- size of the device workspace that
 * fp8_mqa_logits_host needs for an (M, N) problem (H = 32, D = 128), or 0 for a
 * shape outside the contract.
 */
FP8MQA_API uint64_t fp8_mqa_logits_host_workspace_bytes(int64_t M, int64_t N, int32_t H, int32_t D);

/*
 * fp8_mqa_logits_host -- the same operation on HOST buffers.  Enqueues host->device
 * copies of q, k, kv_scale, w, ks, ke into `workspace`, the kernel, and device->host
 * copies of all of out, ordered after the work already on `stream`; work enqueued on
 * `stream` after the call runs after all of it.  The rows go in chunks of about 32 MB of
 * logits (at most 8): the inputs travel on a library stream, the chunks' kernels run on
 * `stream`, and each chunk's logits go back on a second library stream as soon as its
 * kernel is done, so the copies in both directions and the kernels overlap.  The two
 * library streams and their events are created on a device's first call and live until
 * the process exits; calls on one device enqueue one at a time, and their copies share
 * the library streams.  The call can be captured into a CUDA graph (the library streams
 * fork from `stream` by an event and join it again).  Host buffers should be pinned
 * (cudaHostAlloc) for the copies to be asynchronous; pageable memory works but the
 * copies then block.  The call returns after enqueueing; synchronize `stream` before
 * reading `out`.  With clean_logits = 0, the device copy of out is first filled from the
 * host `out`, so untouched entries come back unchanged.
 *   workspace        device pointer, 256-byte aligned, at least
 *                    fp8_mqa_logits_host_workspace_bytes(M, N, H, D) bytes, caller-owned.
 *   workspace_bytes  its size.
 * Other arguments as for fp8_mqa_logits.
 */
FP8MQA_API int fp8_mqa_logits_host(const uint8_t* q_fp8, const uint8_t* k_fp8, const float* kv_scale,
                        const float* w, const int32_t* ks, const int32_t* ke, float* out,
                        int64_t M, int64_t N, int32_t H, int32_t D, int32_t clean_logits,
                        int32_t split_n, void* workspace, uint64_t workspace_bytes,
                        void* stream);

/*
 * fp8_mqa_logits_noalloc -- fp8_mqa_logits for callers that cannot allocate device
 * memory.  The pages this library follows have no counterpart: it exists for hosts such
 * as serving engines that reserve nearly all HBM for their own pools up front and forbid
 * allocations outside them, plug-in interfaces of inference runtimes whose contract bars
 * a plug-in from allocating, and latency-critical loops where a cudaMalloc (which can
 * synchronize the device) or a first-call allocation is not acceptable.
 *
 * Arguments, layouts, results and errors are those of fp8_mqa_logits; the output is the
 * same bit for bit.  Differences:
 *   - It calls no cudaMalloc, cudaFree or other allocating routine.  Its scratch (the
 *     scheduler's work counters and a status word) is a 256-byte device array compiled
 *     into the library, which every GPU that loads the library holds until process exit.
 *     The scratch a call needs does not depend on M or N; a call that needed more than
 *     the array holds would be refused with FP8MQA_ERR_UNSUPPORTED_SHAPE.
 *   - The first call on a device looks up the array's device address (once per device,
 *     with that device current); make that first call before any stream capture.
 *   - Every call shares the one array.  Each call clears the work counters on `stream`
 *     before its kernel, so calls that overlap on the GPU (for example on two streams
 *     at once) race on them and may produce wrong output: order such calls on one
 *     stream or with events.
 *   - A bounded on-device wait that gives up is recorded in the array's status word;
 *     fp8_mqa_logits_check_error reads and clears it (and allocates nothing).
 */
FP8MQA_API int fp8_mqa_logits_noalloc(const uint8_t* q_fp8, const uint8_t* k_fp8,
                                      const float* kv_scale, const float* w, const int32_t* ks,
                                      const int32_t* ke, float* out, int64_t M, int64_t N,
                                      int32_t H, int32_t D, int32_t clean_logits,
                                      int32_t split_n, void* stream);

/*
 * fp8_mqa_topk -- per-row top-k over a logits matrix, the step that consumes the indexer
 * logits (ROCm/aiter PR #7183 "[HIP] [JIT] Add gfx950 prefill FP8 MQA logits", "Test plan":
 * top-512 selections compared end to end; ROCm/aiter PR #6159 "[Triton/Gluon] GFX950 sparse
 * mla optimizations", "Technical Details": sparse MLA with top-k 512).  The pages fix no tie
 * rule or padding; this library reads the step as:
 *   - only finite entries are eligible (-inf, a key outside the row's window, never is);
 *   - row m's result lists its k largest eligible entries by value, descending, and equal
 *     values by index, ascending (-0.0 equals +0.0);
 *   - slots past the row's eligible entries hold index -1 and value -inf.
 * The result is therefore unique.
 *
 *   logits   DEVICE float32, row m at logits + m * ld (ld >= N), 4-byte aligned; typically
 *            the `out` of fp8_mqa_logits with clean_logits = 1.  Not modified.
 *   M, N     rows and entries per row (M >= 0, 0 <= N <= 2^30).  M = 0 enqueues nothing.
 *   k        1 <= k <= 2048.
 *   indices  DEVICE int32 [M, k], row-major, 4-byte aligned, written.
 *   values   DEVICE float32 [M, k] or NULL; when given, the selected logits (their exact
 *            bits), -inf in padded slots.
 *   stream   cudaStream_t; asynchronous.
 * Errors: FP8MQA_ERR_INVALID_ARG (sizes, k, null pointers), FP8MQA_ERR_UNSUPPORTED_SHAPE
 * (N too large), FP8MQA_ERR_MISALIGNED, FP8MQA_ERR_ARCH, FP8MQA_ERR_LAUNCH.  The first call on
 * a device sets up the same per-device state as fp8_mqa_logits.
 */
FP8MQA_API int fp8_mqa_topk(const float* logits, int64_t M, int64_t N, int64_t ld, int32_t k,
                            int32_t* indices, float* values, void* stream);

/*
 * fp8_mqa_topk_windowed -- fp8_mqa_topk restricted to each row's key window: row m's result
 * is the top-k of logits[m, n] for n in [ks[m], ke[m]) (clamped to [0, N); empty when
 * ks[m] >= ke[m]), with the same order, tie rule and padding.  Entries outside the window are
 * never read, so the logits may come from fp8_mqa_logits with clean_logits = 0 (whatever lies
 * outside the windows is ignored), and only the windows' bytes are read.  With the windows that
 * made the logits, the result equals fp8_mqa_topk's on the clean_logits = 1 output.  The page
 * has no such entry; it is this library's way to let the consumer skip the -inf fill.
 *
 *   ks, ke   DEVICE int32 [M], 4-byte aligned, the same windows as fp8_mqa_logits takes; both
 *            null gives fp8_mqa_topk.  Not modified.
 *   the other arguments and the errors are fp8_mqa_topk's; ks without ke (or the reverse) is
 *   FP8MQA_ERR_INVALID_ARG.
 */
FP8MQA_API int fp8_mqa_topk_windowed(const float* logits, int64_t M, int64_t N, int64_t ld,
                                     const int32_t* ks, const int32_t* ke, int32_t k,
                                     int32_t* indices, float* values, void* stream);

/*
 * fp8_mqa_topk_ex -- fp8_mqa_topk_windowed with flags.
 *
 *   flags    0, or FP8MQA_TOPK_UNSORTED: each row's result holds the same entries (the same
 *            set of indices, each with its exact value), in an unspecified order that may differ
 *            between calls; the padding still follows the selected entries.  This skips the
 *            winners' sort, for consumers that take the indices as a set (sparse attention
 *            gathers them).  Any other bit is FP8MQA_ERR_INVALID_ARG.
 *   the other arguments and the errors are fp8_mqa_topk_windowed's.
 */
#define FP8MQA_TOPK_UNSORTED 1
FP8MQA_API int fp8_mqa_topk_ex(const float* logits, int64_t M, int64_t N, int64_t ld,
                               const int32_t* ks, const int32_t* ke, int32_t k, int32_t flags,
                               int32_t* indices, float* values, void* stream);

/* ------------------------------------------------------------------------------------------
 * Paged caches: the operators of a serving step around the logits.  New key and value rows
 * are quantised into pages as they are written, packed back for a prompt chunk, scored for
 * the newest tokens straight from the pages, and attended to -- all of them, or the entries
 * that fp8_mqa_topk selected.
 *
 * A cache is `pages` pages of `page_size` token rows of `heads` heads of `dim` values:
 * element (p, r, h, d) of the data lies at data + p*page_stride + r*row_stride +
 * h*head_stride + d (in elements; the values of a row are contiguous), and for E4M3 the row's
 * scale at scale + p*scale_page_stride + r*scale_row_stride + h*scale_head_stride.  An E4M3 row
 * stands for data * scale.  The strides are free, so keys and values may share one tensor
 * ([pages, 2, page_size, heads, dim]) and heads may come before rows.
 *
 * An E2M1 cache holds 4 bits a value: byte j of a row's dim / 2 has value 2j in its low half and value
 * 2j + 1 in its high half, and the data's strides count bytes.  Beside the row's scale there is an E4M3
 * scale for each 16 values (a group), the dim / 16 bytes of a row at groups + p*group_page_stride +
 * r*group_row_stride + h*group_head_stride.  A value stands for data * group * scale.  A row of 128 takes
 * 76 bytes (132 in E4M3).  fp8_mqa_cache_write, fp8_mqa_cache_read and fp8_mqa_attention_paged take such
 * caches; the indexer's keys stay E4M3.
 *
 * Position n of sequence b lies in page table[b*table_stride + n / page_size], row
 * n % page_size.  A table entry outside [0, pages) is a page that is not there: its positions
 * are never read.  Table entries past a sequence's length are not read either.
 *
 * The first paged call on a device sets up its state (kernel attributes and a status word); make
 * it before any stream capture, as for fp8_mqa_logits.  Kernels are launched so that their set-up need
 * not wait for the kernel before them on the stream: it overlaps the page tables', the norms' and the
 * first of an attention call's, which let it in, and begins with the last block's end of the others; what
 * they read and write is ordered as ever.
 *
 * Limits: dim is 64 or 128; data 16-byte aligned with strides of a multiple of 16 bytes; groups and
 * their strides a multiple of dim / 16 bytes;
 * pages * page_size < 2^31; strides are not negative.  Byte offsets are 64-bit throughout;
 * fp8_mqa_attention_paged counts a cache's rows in units of the greatest common divisor of its
 * page and row strides, of which a cache may span up to 2^32 - 2 (64 GB even at 16 bytes); for E2M1
 * caches the groups and the scales too, whose strides are not negative either.
 * ------------------------------------------------------------------------------------------ */

/* Element types. */
#define FP8MQA_E4M3 0
#define FP8MQA_BF16 1
#define FP8MQA_F16 2
#define FP8MQA_F32 3
#define FP8MQA_E2M1 4 /* 4 bits: 0, 0.5, 1, 1.5, 2, 3, 4 and 6 with a sign */

typedef struct fp8mqa_cache {
    void* data;          /* DEVICE */
    float* scale;        /* DEVICE; NULL unless type is FP8MQA_E4M3 or FP8MQA_E2M1 */
    int64_t pages;
    int32_t page_size;
    int32_t heads;
    int32_t dim;
    int32_t type;        /* FP8MQA_E4M3, FP8MQA_BF16, FP8MQA_F16 or FP8MQA_E2M1 */
    int64_t page_stride, row_stride, head_stride;                    /* elements of data */
    int64_t scale_page_stride, scale_row_stride, scale_head_stride;  /* elements of scale */
    /* From here on for FP8MQA_E2M1 alone; with other types these are not read, and need not be there. */
    uint8_t* groups;     /* DEVICE, E4M3 */
    int64_t group_page_stride, group_row_stride, group_head_stride;  /* bytes */
} fp8mqa_cache;

/*
 * fp8_mqa_cache_write -- quantises T token rows and writes them into one or two E4M3 or E2M1 caches.
 *
 * For each token t and head h, with x its `dim` values in fp32:
 *     a = max(max_d |x_d|, 1e-30);  data_d = e4m3(x_d * (448 / a));  scale = a * (1 / 448)
 * each step rounded to fp32, e4m3() to the nearest even, within +-448.  Into E2M1 caches, with m the
 * largest |x_d| of a group,
 *     group = e4m3(m * 448 / a);  data_d = e2m1(x_d * 2688 / (group * a));  scale = a * (1 / 2688)
 * (data_d = 0 where group is 0), where products are rounded to fp32 (they are exact for 16-bit rows) and
 * quotients are those of an fp32 division; e2m1() to the nearest even, within +-6.  A row that holds a
 * NaN or an infinity reads back as NaN, so that it does not pass for data.
 *
 *   slots    DEVICE int32 [T]: page * page_size + row.  A slot outside [0, pages * page_size)
 *            is skipped (padding).  Tokens of one call must not share a slot: what such a row
 *            holds afterwards is unspecified.
 *   x        DEVICE [T, heads, dim] of x_type (BF16, F16 or F32), element (t, h, d) at
 *            t*x_row_stride + h*x_head_stride + d; aligned to its type.
 *   cache    where x goes.
 *   x2, cache2   NULL, or a second tensor (values next to keys) of x's type and its cache,
 *            with cache's type, page_size, heads and dim and the same slots: one launch writes both.
 * T = 0 enqueues nothing.  No workspace, no allocation; may be captured into a graph.
 */
FP8MQA_API int fp8_mqa_cache_write(const int32_t* slots, int64_t T, int32_t x_type, const void* x,
                                   int64_t x_row_stride, int64_t x_head_stride,
                                   const fp8mqa_cache* cache, const void* x2,
                                   int64_t x2_row_stride, int64_t x2_head_stride,
                                   const fp8mqa_cache* cache2, void* stream);

/*
 * fp8_mqa_cache_read -- packs the rows of B sequences, one after the other, out of an E4M3 or E2M1 cache.
 *
 *   table, table_stride, table_cols   DEVICE int32 page table, B rows of table_cols entries.
 *   starts     DEVICE int32 [B + 1], ascending from 0: sequence b's positions 0, 1, ... go to
 *              output rows starts[b] .. starts[b + 1] - 1.
 *   total      output rows (the caller's copy of starts[B]).  Rows past starts[B] are zeroed.
 *   out        DEVICE [total, heads, dim] of out_type, contiguous, 16-byte aligned:
 *              FP8MQA_E4M3: the stored values, with their scales in out_scale [total, heads]
 *              (with heads = 1 the k_fp8 and kv_scale that fp8_mqa_logits takes);
 *              BF16, F16 or F32: data * scale in fp32, rounded to the type (out_scale is NULL);
 *              the only ones for an E2M1 cache (data * group, which is exact, then * scale).
 * Positions on pages that are not there, or past the table, are zero (and their scale).
 * total * heads < 2^31, and a token's row of `out`, all its heads, is 2^34 bytes at most
 * (FP8MQA_ERR_UNSUPPORTED_SHAPE).
 */
FP8MQA_API int fp8_mqa_cache_read(const fp8mqa_cache* cache, const int32_t* table,
                                  int64_t table_stride, int32_t table_cols, const int32_t* starts,
                                  int64_t B, int64_t total, int32_t out_type, void* out,
                                  float* out_scale, void* stream);

/*
 * fp8_mqa_logits_paged -- the indexer logits of each sequence's T newest tokens, from the pages:
 *
 *   out[b*T + t, n] = scale[n] * sum_h relu(q[b,t,h,:] . k[n,:]) * w[b,t,h]
 *                     for n in [0, lens[b] - (T - 1 - t)),   -inf elsewhere (clean_logits = 1)
 *
 * with k and scale the rows of sequence b (token t of the T newest sees the cache up to itself).
 * Positions on pages that are not there are -inf with either clean_logits.  A NaN in a query, a key, a
 * weight or a scale is NaN in the logits that it belongs to (fp8_mqa_topk passes over them).
 *
 *   q_fp8     DEVICE [B, T, H, D] E4M3, contiguous, 16-byte aligned; H = 32, D = 128.
 *   w         DEVICE [B, T, H] float32, contiguous, 16-byte aligned.
 *   keys      the E4M3 cache, heads = 1, dim = 128.
 *   lens      DEVICE int32 [B]: length with the T newest tokens included; <= 0 is an empty
 *             sequence.  Lengths are clamped to N and to table_cols * page_size.
 *   out       DEVICE float32, row r at out + r * ld, N entries a row, 4-byte aligned.
 *             clean_logits = 0: out-of-window entries are not written.
 * The result feeds fp8_mqa_topk as it is.  No workspace, no allocation.
 */
FP8MQA_API int fp8_mqa_logits_paged(const uint8_t* q_fp8, const float* w, int64_t B, int32_t T,
                                    int32_t H, int32_t D, const fp8mqa_cache* keys,
                                    const int32_t* table, int64_t table_stride,
                                    int32_t table_cols, const int32_t* lens, float* out,
                                    int64_t ld, int64_t N, int32_t clean_logits, void* stream);

/*
 * fp8_mqa_attention_paged -- attention of one new token per row over a paged cache:
 *
 *   x_n = sm_scale * q[b,h,:] . k[n,g,:],  out[b,h,:] = sum_n softmax(x)_n v[n,g,:],
 *   lse[b,h] = log sum_n exp(x_n),   g = h / (q_heads / heads)
 *
 * over the positions n in [0, lens[b]), or over those that `indices` lists.  Products are
 * fp32-accumulated; the softmax is fp32; weights are rounded to 16 bits for the second product.
 * A row with no position: out is 0 and lse is -inf.
 *
 *   q         DEVICE [B, q_heads, dim] of q_type (BF16 or F16), element (b, h, d) at
 *             b*q_row_stride + h*q_head_stride + d; 16-byte aligned, strides too.  q_heads is a
 *             multiple of the cache's heads.
 *   k, v      caches of one type, page_size, heads and dim, over one page table: E4M3, E2M1, or q's type.
 *   lens      DEVICE int32 [B]; clamped to [0, table_cols * page_size].
 *             table_cols * page_size, or n_indices, is 2^31 - 1025 at most.  The work is laid out
 *             for rows as long as the table is wide: where all are known to be much shorter, a
 *             smaller table_cols (the table_stride stays) is faster, by up to a fifth.
 *   n_indices -1: each row attends to all of its positions.  Otherwise `indices` is DEVICE int32
 *   indices   with n_indices entries a row, row b at indices + b*indices_stride: the positions that
 *             row b attends to, for all its heads, in any order; entries outside [0, lens[b]) are
 *             ignored (the -1 of fp8_mqa_topk's padding), a position listed twice counts twice.
 *             With a table_stride of 0 the rows share one sequence.
 *   out       DEVICE [B, q_heads, dim] of q_type, contiguous, 16-byte aligned.
 *   lse       NULL, or DEVICE float32 [B, q_heads].
 *   workspace DEVICE, 256-byte aligned, at least fp8_mqa_attention_paged_workspace_bytes(...) bytes;
 *             its content does not matter before or after the call, and calls that may overlap on
 *             the GPU need one each.
 */
FP8MQA_API int fp8_mqa_attention_paged(const void* q, int32_t q_type, int64_t B, int32_t q_heads,
                                       int64_t q_row_stride, int64_t q_head_stride,
                                       const fp8mqa_cache* k, const fp8mqa_cache* v,
                                       const int32_t* table, int64_t table_stride,
                                       int32_t table_cols, const int32_t* lens,
                                       const int32_t* indices, int64_t indices_stride,
                                       int32_t n_indices, float sm_scale, void* out, float* lse,
                                       void* workspace, uint64_t workspace_bytes, void* stream);

/* fp8_mqa_attention_paged_workspace_bytes -- the workspace of a call with q_heads query
 * and kv_heads key heads of width dim, on the current device (0 when there is none of compute
 * capability 10.3).  It does not depend on the rows or their lengths. */
FP8MQA_API uint64_t fp8_mqa_attention_paged_workspace_bytes(int32_t q_heads, int32_t kv_heads,
                                                            int32_t dim);

/* ------------------------------------------------------------------------------------------
 * A step's other operators: its page tables, and what comes between a layer's projection and
 * the caches.
 * ------------------------------------------------------------------------------------------ */

/*
 * fp8_mqa_pages_update -- changes the lengths of B requests, gives and takes their pages, and says where
 * their new tokens go.
 *
 * Request b of length n holds the pages table[b*table_stride + c], c < ceil(n / page_size).  The pages
 * that nobody holds are the first *n_free entries of free_pages, a stack.  With to = max(0, lens[b] +
 * change[b]):
 *   1. requests with change < 0 shrink; the pages that they need no more go onto the stack, in the order
 *      of requests and of columns (what does not go into `capacity` entries is dropped);
 *   2. the others grow; the pages that they need go from the top of the stack into their row, in the same
 *      order.  A request that needs more than table_cols pages does not fit.  From the first request on
 *      for which the stack is too short, requests that need new pages do not fit either (those that stay
 *      on their last page do).  One that does not fit keeps its length and takes nothing;
 *   3. lens and *n_free are brought up to date.
 * Table entries past a request's length, and entries of free_pages past *n_free, are left as they are.
 *
 *   table       DEVICE int32, written; rows do not overlap (table_stride >= table_cols).
 *   lens        DEVICE int32 [B], written; values are taken within [0, table_cols * page_size].
 *   change      DEVICE int32 [B]: 1 or more for a decode step, a prompt chunk's tokens, minus the length
 *               for a request that ends, minus the drafted tokens that were not accepted, 0 for nothing.
 *   free_pages, capacity, n_free   DEVICE int32 [capacity], written, and its count, DEVICE int32, written.
 *   total       rows of the three arrays below; rows past starts[B] are padding, tokens past `total`
 *               have no row.
 *   slots       DEVICE int32 [total]: where fp8_mqa_cache_write puts each new token, request after
 *               request; -1 for those of a request that does not fit, and for padding.
 *   positions   DEVICE int32 [total]: each new token's position in its request (0 for padding).
 *   rows        DEVICE int32 [total]: each new token's request (0 for padding).
 *   starts      DEVICE int32 [B + 1]: request b's new tokens are rows starts[b] .. starts[b + 1] - 1 (sums
 *               stop at 2^31 - 1).
 *   changed     DEVICE int32 [B]: by how much the length changed (0 for a request that does not fit).
 * Limits: B <= 8192, table_cols * page_size < 2^31, B * table_cols < 2^31 (FP8MQA_ERR_UNSUPPORTED_SHAPE).
 * Arrays that overlap are refused (FP8MQA_ERR_INVALID_ARG).
 * The result is always the same for the same arguments.  No workspace, no allocation; may be captured
 * into a graph.
 */
FP8MQA_API int fp8_mqa_pages_update(int32_t* table, int64_t table_stride, int32_t table_cols,
                                    int32_t page_size, int32_t* lens, const int32_t* change,
                                    int64_t B, int32_t* free_pages, int64_t capacity,
                                    int32_t* n_free, int64_t total, int32_t* slots,
                                    int32_t* positions, int32_t* rows, int32_t* starts,
                                    int32_t* changed, void* stream);

/* Rows [T, heads, dim] of a tensor and where their results go; strides in elements. */
typedef struct fp8mqa_heads {
    const void* x;        /* DEVICE, aligned to its type */
    const void* weight;   /* DEVICE [dim], or NULL: rows are not normed */
    void* out;            /* DEVICE, aligned to its type (E4M3: to 4 bytes, strides too); may be x itself,
                             with x's strides, where the type is x's, and else shares no memory with
                             anything that the call reads or writes */
    float* out_scale;     /* DEVICE [T, heads] for E4M3 results, else NULL */
    int64_t row_stride, head_stride;
    int64_t out_row_stride, out_head_stride;
    int32_t heads;
    int32_t weight_type;  /* x's, or FP8MQA_F32 */
} fp8mqa_heads;

/*
 * fp8_mqa_norm_rotate -- norms each head of queries and keys and rotates it by its token's position.
 *
 *     y = x * (mean_d(x_d^2) + eps)^-1/2 * weight       (y = x without a weight)
 *     out_a = y_a cos t - y_b sin t,  out_b = y_b cos t + y_a sin t,   t = positions[token] * inv_freq[i]
 *
 * for the pairs i < rotated / 2 of the first `rotated` values: (a, b) = (i, i + rotated / 2), or
 * (2i, 2i + 1) with interleaved = 1; the other values are y.  All in fp32, rounded once to x's type, or to
 * E4M3 with a scale a row as fp8_mqa_cache_write does: the q_fp8 of fp8_mqa_logits with dim 128, whose scales
 * the caller multiplies into w.  Sums of squares are fp32 and want values under 10^18.  However many turns t
 * is, it is off by little more than 2^-26 of a turn and by the frequency's own error, (1 + |f|) 2^-64 turns
 * for f turns a position, times |position|: as exact as fp32 holds a turn up to positions of 2^39, not beyond.
 *
 *   q, k        the tensors; k may be NULL, and heads 0.
 *   x_type      FP8MQA_BF16, FP8MQA_F16 or FP8MQA_F32, of both.  out_type: x_type or FP8MQA_E4M3.
 *   dim         64 or 128.  rotated: a multiple of 16, at most dim; 0 only norms.
 *   positions   DEVICE int32 or int64 [T] (position_bytes 4 or 8); any value, negative ones too.
 *   inv_freq    DEVICE float32 [rotated / 2], radians a position; where one is not finite its pair is NaN.
 * T * (all heads) < 2^31.  Results that share memory with one another or with an argument, but for x
 * itself, are refused (FP8MQA_ERR_INVALID_ARG; slices of one tensor do not share it, but many rows that lie
 * between one another's at different strides are refused too).  No workspace, no allocation; may be captured
 * into a graph.
 */
FP8MQA_API int fp8_mqa_norm_rotate(const fp8mqa_heads* q, const fp8mqa_heads* k, int32_t x_type,
                                   int32_t out_type, int64_t T, int32_t dim,
                                   const void* positions, int32_t position_bytes,
                                   const float* inv_freq, int32_t rotated, int32_t interleaved,
                                   float eps, void* stream);

/* fp8_mqa_logits_strerror -- a static, human-readable name for a status code. */
FP8MQA_API const char* fp8_mqa_logits_strerror(int status);

#ifdef __cplusplus
}
#endif

#endif /* FP8_MQA_LOGITS_H */
