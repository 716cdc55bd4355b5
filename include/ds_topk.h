/*
 * ds_topk.h -- C ABI of the GB300 DeepSelect row-wise top-k library (libds_topk.so).
 *
 * The operation is DeepSelectTopk as defined in DeepSelect-deep-dive.md ("Algorithm"):
 * for every row of N scores, keep a threshold T (initially -inf), visit the row in
 * blocks of B elements in a random block order that does not depend on the data,
 * append every element greater than T to an on-chip candidate buffer, and when the
 * buffer holds at least k + B2 entries after a block, shrink it back to its k largest
 * entries (RadixSelectTopK) and set T to the smallest of them.  A final RadixSelectTopK
 * returns k values and their int32 column indices.  The split-row mode that spreads one
 * row over several CTAs and merges their candidates follows the same page's
 * "Implementation" section (thread-block cluster paragraph).
 *
 * Order of values.  Values are compared by their IEEE bit patterns mapped to an
 * order-preserving unsigned key (sign set: invert all bits; sign clear: set the sign
 * bit), the mapping the DeepSelect TopK tutorial (section 4.6) uses for radix
 * selection.  This is a total order: -NaN < -inf < ... < -0 < +0 < ... < +inf < +NaN.
 *
 * Block order.  Block b of row r is visited in the order of
 *   u_b = Philox4x32-10(key = (seed & 0xffffffff, seed >> 32), counter = (b, r, 0, 0))[0]
 * ascending, ties by b (Salmon et al., "Parallel Random Numbers: As Easy as 1, 2, 3",
 * SC'11).  When a row is split into P parts, part p takes every P-th block from block p
 * (blocks p, p + P, p + 2P, ...) and visits them in the order of the same draws.
 *
 * Results.  out_vals[r*k + j] / out_idx[r*k + j], j < k, hold the k largest values of
 * row r (bit copies of the input) and their columns, in no particular order (in order of
 * value descending, equal values by column ascending, with ds_options.sorted).  Among
 * values equal to the k-th largest, which columns are returned is unspecified; the
 * value multiset is always exact.
 *
 * All calls are asynchronous on `stream` and return once the work is enqueued.  Errors
 * found on the host are returned before anything is launched.  Errors found on the
 * device (a bounded wait that ran out) are recorded in a per-device status word that
 * ds_get_device_status() reads.  Nothing here allocates memory except ds_topk() when a
 * row is split over more than one cluster (see ds_topk_ex).
 */
#ifndef DS_TOPK_H
#define DS_TOPK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same declaration as the CUDA runtime's; a cudaStream_t may be passed directly. */
typedef struct CUstream_st* cudaStream_t;

typedef enum {
    DS_BF16 = 0, /* 16-bit bfloat16, passed as raw 16-bit patterns */
    DS_FP32 = 1  /* 32-bit IEEE float */
} ds_dtype;

typedef enum {
    DS_OK = 0,
    DS_ERR_INVALID_ARG = 1, /* null pointer, rows < 0, N < 1, k < 1, k > N, B < 0, B2 < 0,
                               row_stride < N, unknown dtype                          */
    DS_ERR_ALIGNMENT = 2,   /* x, out_vals or out_idx not 16-byte aligned, or (rows > 1)
                               row_stride * sizeof(element) not a multiple of 16       */
    DS_ERR_UNSUPPORTED = 3, /* k > 4096, N >= 2^31, B * sizeof(element) not a multiple of
                               16, or the candidate buffer (k + B + B2 entries) and the
                               copy ring do not fit in one SM's shared memory         */
    DS_ERR_CUDA = 4,        /* a CUDA runtime call failed (launch, attribute, alloc)    */
    DS_ERR_TIMEOUT = 5,     /* a bounded device-side wait ran out (ds_get_device_status) */
    DS_ERR_INTERNAL = 6,    /* a device-side consistency check failed                   */
    DS_ERR_WORKSPACE = 7    /* caller workspace too small, or would allocate while the
                               stream is being captured                               */
} ds_status;

/* Number of int64 statistics per row written by ds_topk_ex (options.stats). */
#define DS_NSTAT 8
/* statistics layout, per row: A (elements appended), R (in-loop compactions),
   W (total input size of all compactions, the final one included), max |C|,
   m = ceil(N/B), 0, R, 0 -- the quantities of the expected-work analysis of
   DeepSelect-deep-dive.md ("Expected Upper Bound"). */

/*
 * ds_topk -- row-wise top-k of `rows` rows.
 *   x           device pointer; row r starts at element r*row_stride.  16-byte aligned.
 *   dtype       DS_BF16 or DS_FP32.
 *   rows        number of rows (0: nothing is done, DS_OK).
 *   N           elements per row, 1 <= N < 2^31.
 *   row_stride  elements between row starts, >= N; when rows > 1, row_stride*sizeof(element)
 *               must be a multiple of 16 bytes (1024 recommended).
 *   k           1 <= k <= min(N, 4096).
 *   B, B2       block size and compaction slack of the method (>= 1), or 0 for the
 *               library's choice: B = 8192 when the rows fit one wave of CTAs
 *               (ceil(rows / SMs) == 1) and 4096 otherwise, B2 = 4096 -- the shipped
 *               CUDA configuration the DeepSelect TopK tutorial describes (section 4.7);
 *               ds_get_plan reports the values in effect.  B*sizeof(element) must be a
 *               multiple of 16 bytes, k + B + B2 <= 2^20, and one CTA visits at most 1024
 *               blocks (with one CTA per row: ceil(N/B) <= 1024).
 *   seed        selects the block order (see above).
 *   out_vals    device, rows*k elements of dtype; 16-byte aligned.  Caller-owned.
 *   out_idx     device, rows*k int32; 16-byte aligned.  Caller-owned.
 *   stream      CUDA stream (0 = legacy default stream).
 * The library chooses how many CTAs share a row: rows split over a cluster, or rows
 * that already fill the GPU one per CTA, run the split-row kernel (warm-up threshold
 * from a sample of the row, compaction when a chunk's survivors do not fit; rows held
 * whole in one cluster start from a speculative threshold, checked and redone when it
 * was too high -- ds_plan.spec_k); only ds_topk_ex with parts = 1 runs the pages'
 * one-CTA schedule exactly.  Results are exact on every path.  When a row is
 * split over more than one thread-block cluster it uses a library-owned workspace, one
 * per (device, stream) -- per thread as well for cudaStreamPerThread -- so calls on
 * different streams may run concurrently.  It is grown with cudaMalloc (and cleared with
 * cudaMemsetAsync on `stream`) on a call that is not being stream-captured; a call under
 * capture that would need to grow it returns DS_ERR_WORKSPACE.  An outgrown workspace is
 * kept, not freed, until the process exits (launches already enqueued may still use it),
 * so growing never synchronises the device.  Launches let the
 * next kernel on the stream start as this one's CTAs leave (programmatic dependent
 * launch); a call reads x only once the kernel before it has completed (see
 * ds_options.input_ready).
 */
ds_status ds_topk(const void* x, int32_t dtype, int64_t rows, int64_t N, int64_t row_stride,
                  int32_t k, int32_t B, int32_t B2, uint64_t seed, void* out_vals,
                  int32_t* out_idx, cudaStream_t stream);

typedef struct {
    int32_t parts;          /* CTAs per row: 0 = library choice; 1 = one CTA per row (the
                               pages' schedule, required for stats); P > 1 splits each
                               row's blocks into P interleaved sets (block b to part
                               b mod P)                                               */
    int32_t cluster;        /* CTAs per thread-block cluster (divides parts, <= 16);
                               0 = library choice                                     */
    int64_t* stats;         /* optional device array rows*DS_NSTAT, parts == 1 only    */
    void* workspace;        /* optional caller-owned device workspace; NULL = library  */
    size_t workspace_bytes; /* its size; see ds_workspace_bytes                        */
    int32_t input_ready;    /* 0 (default): the call reads x only after every earlier
                               kernel on the stream has completed, so x may be written
                               by the kernel just before it.  Nonzero: the caller states
                               that x was complete before that kernel started, and the
                               call starts reading x while that kernel is still running
                               (consecutive calls on static inputs overlap their edges) */
    int32_t sorted;         /* nonzero: each row's k results in order of value descending
                               (the key order above), equal values by column ascending
                               -- the pages' sorted_value flag; a second kernel sorts the
                               k results of each row in shared memory at the end      */
} ds_options;

/* ds_topk with explicit options (NULL = defaults, identical to ds_topk). */
ds_status ds_topk_ex(const void* x, int32_t dtype, int64_t rows, int64_t N, int64_t row_stride,
                     int32_t k, int32_t B, int32_t B2, uint64_t seed, void* out_vals,
                     int32_t* out_idx, const ds_options* options, cudaStream_t stream);

/* The launch the library would use for these arguments (host only, no launch). */
typedef struct {
    int32_t parts;          /* CTAs per row                                            */
    int32_t cluster;        /* CTAs per cluster                                        */
    int32_t threads;        /* threads per CTA                                         */
    int32_t chunk_elems;    /* elements per bulk copy                                  */
    int32_t stages;         /* depth of the copy ring                                  */
    int32_t capacity;       /* candidate-buffer entries: k + B + B2 for rows of one CTA;
                               at least k + one chunk for split rows, widened into the
                               shared memory the layout leaves over                    */
    int64_t smem_bytes;     /* dynamic shared memory per CTA                           */
    int64_t workspace_bytes;/* device workspace needed (0 unless split over clusters)  */
    int32_t ctas_per_sm;    /* resident CTAs per SM for this configuration             */
    int32_t merge_launch;   /* 1 when a second (merge) kernel runs                      */
    int32_t B;              /* block size in effect (the library's choice when 0 was passed) */
    int32_t B2;             /* compaction slack in effect (likewise)                   */
    int32_t spec_k;         /* rows held whole in one cluster: the first attempt filters
                               from an estimate of the spec_k-th largest sampled group
                               maximum, a threshold nothing proves; the final select
                               checks that k keys reach it and otherwise filters the
                               row's chunks, still in shared memory, from the proven
                               threshold (0 = no speculation)                          */
} ds_plan;

/* Errors as ds_topk's host checks (DS_ERR_INVALID_ARG, DS_ERR_UNSUPPORTED), and
   DS_ERR_CUDA when no device can be queried.  Without a device, the environment variable
   DS_PLAN_DEVICE="sms,smem_optin,smem_per_sm" (SM count and the two shared-memory limits
   in bytes) describes one, for planning only; launches still need the real device. */
ds_status ds_get_plan(int32_t dtype, int64_t rows, int64_t N, int32_t k, int32_t B, int32_t B2,
                      const ds_options* options, ds_plan* plan);

/* Workspace bytes ds_topk_ex needs for these arguments (0 when none). */
ds_status ds_workspace_bytes(int32_t dtype, int64_t rows, int64_t N, int32_t k, int32_t B,
                             int32_t B2, const ds_options* options, size_t* bytes);

/*
 * ds_topk_sample -- top-k sampling, the sampler use of top-k (DeepSelect TopK tutorial,
 * section 1.1: at sampling time top-k picks the candidate tokens out of the vocabulary's
 * logits).  Per row: the k largest logits, sorted as with ds_options.sorted (value
 * descending, equal values by column ascending), are written to out_vals / out_idx as by
 * ds_topk_ex; candidate i gets weight w_i = exp((v_i - v_0) / temperature); the row's
 * token is out_idx[row*k + j] for the first j whose running sum w_0 + ... + w_j exceeds
 * uniforms[row] * (w_0 + ... + w_{k-1}) (the last candidate if rounding leaves none), and
 * out_prob[row] = w_j / (sum of all w).  Weights and sums are fp32, summed in candidate
 * order.
 *   logits, dtype .. seed, out_vals, out_idx   as ds_topk (B = 0 / B2 = 0 allowed)
 *   temperature  > 0 and finite, else DS_ERR_INVALID_ARG
 *   uniforms     device, rows floats in [0, 1): the caller's random draws (one per row)
 *   out_token    device, rows int32: the sampled column of each row
 *   out_prob     device, rows floats, or NULL: the sampled candidate's probability
 * Logits are expected finite (an infinite or NaN logit makes the weights undefined; the
 * top-k part is exact for any values).  Asynchronous on `stream`.
 */
ds_status ds_topk_sample(const void* logits, int32_t dtype, int64_t rows, int64_t N, int64_t row_stride,
                         int32_t k, int32_t B, int32_t B2, uint64_t seed, float temperature,
                         const float* uniforms, void* out_vals, int32_t* out_idx, int32_t* out_token,
                         float* out_prob, cudaStream_t stream);

/* Synchronizes `stream`, then reads and clears the calling device's status word:
   DS_OK, DS_ERR_TIMEOUT or DS_ERR_INTERNAL. */
ds_status ds_get_device_status(cudaStream_t stream);

/* Static description of a status code. */
const char* ds_status_string(ds_status status);

/* Library version, e.g. "ds_topk 0.1 sm_103a". */
const char* ds_version(void);

/* The block visiting order the scan kernel uses (see "Block order" above), computed on
 * the device by the same code: out_perm[i] (device, nblocks int32) = the i-th block
 * visited among blocks first_block .. first_block+nblocks-1 of `row`.
 * 1 <= nblocks <= 1024.  For parity checks of the block order; asynchronous on stream. */
ds_status ds_block_order(uint64_t seed, int64_t row, int64_t first_block, int32_t nblocks,
                         int32_t* out_perm, cudaStream_t stream);

/* Runs one bounded wait on an mbarrier phase that never completes, with a limit of
 * `cycles` SM clock cycles (0 .. 2e9).  The wait runs out, the kernel records
 * DS_ERR_TIMEOUT in the device status word and returns; ds_get_device_status() then
 * reports it.  Checks the failure path of the device-side waits without a GPU fault. */
ds_status ds_wait_probe(int64_t cycles, cudaStream_t stream);

/*
 * ds_topk_noalloc -- ds_topk_ex for callers that cannot allocate device memory.
 *
 * This entry point has no counterpart in the pages; it exists for callers that may not
 * call cudaMalloc: code that runs while a CUDA graph is being captured (where an
 * allocation would break or escape the capture), serving loops that forbid allocator
 * calls because cudaMalloc/cudaFree can synchronise the device and stall other work,
 * and processes whose caching allocator has already reserved nearly all device memory.
 *
 * Arguments are those of ds_topk_ex, with `parts` and `cluster` as in ds_options
 * (0 = library choice).  When the launch needs scratch memory (a row split over more
 * than one thread-block cluster) it uses a fixed array compiled into the library's
 * device image instead of a workspace: at most ds_noalloc_scratch_bytes() bytes
 * (4 MiB; about rows * clusters_per_row * k * 8 bytes are needed); a launch that would
 * need more returns DS_ERR_WORKSPACE.  The array exists on every device that loads the
 * library until the process exits.  It calls no cudaMalloc, cudaFree or allocating
 * library routine.
 *
 * The first call on a device that needs the scratch looks up its device address (with
 * that device current); make that first call before any stream capture.  The address is
 * kept per device index for the life of the process: after cudaDeviceReset (or with a
 * different primary context for that device) the kept address is stale, so such a
 * process must not call this entry point again on that device.  All calls
 * share the one array: calls whose work overlaps on the GPU (for instance on different
 * streams) race on it and must be ordered by the caller.
 */
ds_status ds_topk_noalloc(const void* x, int32_t dtype, int64_t rows, int64_t N,
                          int64_t row_stride, int32_t k, int32_t B, int32_t B2, uint64_t seed,
                          void* out_vals, int32_t* out_idx, int32_t parts, int32_t cluster,
                          cudaStream_t stream);

/* Size of the fixed scratch array ds_topk_noalloc uses, in bytes. */
size_t ds_noalloc_scratch_bytes(void);

/* ======================================================================================
 * Operators around the top-k in a decoding step: the experts' gate, the verification of
 * drafted tokens, and a key/value cache in 4 bits with the attention that reads it.
 *
 * As above: calls are asynchronous on `stream`, errors found on the host are returned before
 * anything is launched, inputs and outputs are caller-owned memory of the current device, which
 * `stream` belongs to (the Python functions make their tensors' device current), and a call may be
 * captured in a graph (ds_cache_attention with the library's workspace once it has run on that
 * stream with arguments that need as much, see there).  Launches are programmatic dependent ones: a kernel
 * touches memory only once the kernel before it on the stream has completed.
 * Pointers are aligned to their element unless a call says otherwise (DS_ERR_ALIGNMENT).
 * Logits, keys, values and queries are expected finite, -inf in logits excepted; other values
 * give undefined numbers in their own rows, never a fault.
 * ==================================================================================== */

typedef enum { DS_SOFTMAX = 0, DS_SIGMOID = 1 } ds_scoring;
typedef enum { DS_GROUP_MAX = 0, DS_GROUP_TOP2 = 1 } ds_group_score;

/*
 * ds_route -- the gate of a mixture of experts: each row's k best experts and their weights.
 * Scores of a row x of E logits: s = softmax(x) (DS_SOFTMAX) or 1 / (1 + exp(-x)) (DS_SIGMOID).
 * Choice values: s + bias, or x itself without a bias (s rises with x).  groups > 1: experts
 * lie in `groups` runs of E / groups; a run's score is its largest choice value (DS_GROUP_MAX)
 * or the sum of its two largest (DS_GROUP_TOP2; without a bias of its two largest s), and only
 * experts of the topk_groups best runs are eligible.  The k eligible experts of the largest
 * choice values are returned in descending order; every tie, of experts or groups, goes to the
 * lower index, and -0 equals +0.  weight_j = scale * s_j / (renormalise ? sum of the k s : 1);
 * a sum of 0 gives weights of 0.  The bias moves the choice only.  The softmax's sum takes
 * exponentials that are off by 2^-22 of each; the chosen scores themselves go by expf.
 *   logits, dtype   row r starts at element r * row_stride (any stride >= E)
 *   rows            >= 0
 *   E, k            1 <= k <= min(E / groups * topk_groups, 32); E <= 512, groups <= 32
 *   bias            E floats, or NULL
 *   out_weights     rows * k floats;  out_experts  rows * k int32
 *   counts          E int32 or NULL: the number of rows that chose each expert is ADDED to it
 */
ds_status ds_route(const void* logits, int32_t dtype, int64_t rows, int32_t E, int64_t row_stride, int32_t k,
                   int32_t scoring, const float* bias, int32_t groups, int32_t topk_groups, int32_t group_score,
                   int32_t renormalise, float scale, float* out_weights, int32_t* out_experts, int32_t* counts,
                   cudaStream_t stream);

/*
 * ds_route_backward -- gradient of ds_route's weights with respect to its logits, given the
 * experts it chose (the choice is held constant, so the bias has no gradient).
 *   grad_weights    rows * k floats
 *   experts         rows * k int32, distinct within a row; an index outside [0, E) has no part
 *   grad_logits     rows of E elements of dtype, row r at element r * grad_stride (>= E);
 *                   every element is written; must not overlap logits
 */
ds_status ds_route_backward(const float* grad_weights, const void* logits, int32_t dtype, int64_t rows, int32_t E,
                            int64_t row_stride, int32_t k, const int32_t* experts, int32_t scoring,
                            int32_t renormalise, float scale, void* grad_logits, int64_t grad_stride,
                            cudaStream_t stream);

/*
 * ds_verify_drafts -- speculative sampling's verification, per sequence b.
 * Place i = 0 .. S has target logits x_i (the row after i accepted drafts), p_i =
 * softmax(x_i / temperature), one-hot at the first maximum where the temperature is <= 0.
 * Draft i (token t_i, drawn from q_i) is accepted iff drafts 0 .. i-1 were and
 * uniforms[b, i] * q_i(t_i) < p_i(t_i).  At the first draft that is not accepted, or after the
 * sequence's last draft, one more token is emitted: argmax_v r_v / noise[b, v], with
 * r = max(p_i - q_i, 0) at a refused draft (p_i if that is 0 everywhere) and r = p_i after the
 * last; ties to the lowest v.  With exponential noise the tokens are distributed as samples
 * of the target.  Sums and the race take exponentials that are off by 2^-22 of each (probabilities of
 * 129280 logits come out within 2.4e-7).
 *   logits, dtype    place i of sequence b starts at element b * seq_stride + i * row_stride;
 *                    -inf excludes a token.  A row of -inf alone: refused, token -1, probability 0
 *   sequences        >= 0; drafts_per_sequence S >= 0 (<= 1024); 1 <= V <= 2^30
 *   drafts           [sequences, S] int32; a token outside [0, V) is refused
 *   draft_lens       [sequences] int32 drafts of each sequence (clamped to 0 .. S), or NULL: S
 *   draft_probs      q, floats, draft i of sequence b at b * probs_seq_stride + i *
 *                    probs_row_stride; NULL: q_i is one-hot at t_i (a looked-up draft)
 *   uniforms         [sequences, S] floats in [0, 1)
 *   noise            [sequences, V] positive floats, sequence b at b * noise_stride: independent
 *                    draws of the exponential distribution
 *   temperatures     [sequences] finite floats, or NULL: `temperature` (>= 0, finite) for all
 *   out_tokens       [sequences, S + 1] int32: the accepted drafts, the emitted token, then -1
 *   out_accepted     [sequences] int32: the number of accepted drafts
 *   out_probs        [sequences, S + 1] floats or NULL: p_i of each token, 0 after the last
 */
ds_status ds_verify_drafts(const void* logits, int32_t dtype, int64_t sequences, int32_t drafts_per_sequence,
                           int64_t V, int64_t seq_stride, int64_t row_stride, const int32_t* drafts,
                           const int32_t* draft_lens, const float* draft_probs, int64_t probs_seq_stride,
                           int64_t probs_row_stride, const float* uniforms, const float* noise, int64_t noise_stride,
                           const float* temperatures, float temperature, int32_t* out_tokens, int32_t* out_accepted,
                           float* out_probs, cudaStream_t stream);

/*
 * The 4-bit cache.  A key or value row of D numbers x is held as D codes c in 0 .. 15 and a
 * pair (s, m) of bf16, standing for s * c + m:  m = bf16(min x), s = bf16((max x - m) / 15),
 * c = clamp(rint((x - m) / s), 0, 15) (0 where s < 2^-126, negative s included: a row so narrow that
 * m was rounded up past its maximum), the quotients as fp32 products with 1/15 and 1/s.  Numbers up to
 * 2^126 in size come back finite.  Layout, caller-owned:
 *   cache   [pages][heads][page][2][D / 2] bytes, 16-byte aligned: key, then value; number 2 j
 *           in the low half of byte j, 2 j + 1 in the high half
 *   scales  [pages][heads][page][4] bf16, 8-byte aligned: key s, key m, value s, value m
 * page is a power of two, D 64 or 128 (DS_ERR_UNSUPPORTED).  Token slot t is place t % page of
 * page t / page.
 *
 * ds_cache_store writes `tokens` tokens' keys and values (token i, head h at element
 * i * token_stride + h * head_stride; base and strides multiples of 16 bytes) to slots[i]; a
 * slot outside [0, pages * page) is skipped (a padded token).  Slots of one call are distinct.
 * ds_cache_load reads slots back as dtype, [tokens, heads, D] each, 16-byte aligned; a slot
 * outside gives zeros.
 */
ds_status ds_cache_store(const void* k, const void* v, int32_t dtype, int64_t tokens, int32_t heads, int32_t D,
                         int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                         void* cache, void* scales, int64_t pages, int32_t page, const int32_t* slots,
                         cudaStream_t stream);
ds_status ds_cache_load(const void* cache, const void* scales, int64_t pages, int32_t page, const int32_t* slots,
                        int64_t tokens, int32_t heads, int32_t D, int32_t dtype, void* out_k, void* out_v,
                        cudaStream_t stream);

/*
 * ds_cache_attention -- attention of each sequence's newest tokens over the 4-bit cache.
 * Token i of the `tokens` of sequence b sees the positions below lens[b] - (tokens - 1 - i)
 * (its own key and value are stored already), or those of them that its `indices` list:
 *   out = sum_j P_j v_j,  P = softmax_j(scale * q . k_j),  lse = log sum_j exp(scale * q . k_j).
 * Query head h reads key head h / (q_heads / heads).  A token that sees nothing has out 0 and
 * lse -inf.
 *   q, dtype     token i, head h of sequence b at element b * q_seq_stride + i * q_token_stride
 *                + h * q_head_stride, D numbers
 *   table        [sequences, table_width] int32 (row stride table_stride): position j of sequence
 *                b lies in page table[b, j / page]; a position whose page is outside [0, pages)
 *                is not seen
 *   lens         [sequences] int32, clamped to 0 .. table_width * page
 *   indices      [sequences, tokens, K] int32 positions (as ds_topk returns them), or NULL; one
 *                outside the visible positions (-1 as padding) is not seen, one listed twice
 *                counts twice; K = 0 with any non-null pointer is a list of nothing, of which
 *                nothing is read
 *   scale        finite;  out  [sequences, tokens, q_heads, D] dtype, 16-byte aligned;  out_lse  [sequences,
 *                tokens, q_heads] floats or NULL
 * Results are finite for |q| < 2^113, |v| <= 2^90 and products scale q_d k_d up to 2^100; any number
 * elsewhere affects only the rows that see it.
 * q enters in its own precision, scores, softmax sums and outputs are summed in fp32; the weights
 * that meet the values are rounded to 11 bits for bf16 q and 22 for fp32.  Positions are split
 * over CTAs whose partial results lie in a library-owned workspace of (device, stream), grown with
 * cudaMalloc as ds_topk's is: a call under stream capture that would have to grow it returns
 * DS_ERR_WORKSPACE, and graphs captured on one stream share it, so that they must not run at the same
 * time.  ds_cache_attention_ex takes the caller's workspace instead.  pages >= 1, table_width >= 1,
 * pages * page * heads < 2^32 - 1, table_width * page <= 2^30, K <= 2^30.
 */
ds_status ds_cache_attention(const void* q, int32_t dtype, int64_t sequences, int32_t tokens, int32_t q_heads,
                             int32_t D, int64_t q_seq_stride, int64_t q_token_stride, int64_t q_head_stride,
                             const void* cache, const void* scales, int64_t pages, int32_t heads, int32_t page,
                             const int32_t* table, int64_t table_width, int64_t table_stride, const int32_t* lens,
                             const int32_t* indices, int32_t K, float scale, void* out, float* out_lse,
                             cudaStream_t stream);

/*
 * ds_cache_attention_ex -- ds_cache_attention with the caller's workspace: device memory, 16-byte
 * aligned, of at least ds_cache_attention_workspace_bytes() bytes (else DS_ERR_WORKSPACE), with any
 * content, not used by anything else until the call's work is done.  NULL: the library's.  (The
 * Python function takes it from torch's allocator.)
 * ds_cache_attention_workspace_bytes -- the bytes a call of these sizes needs on the current device,
 * 0 for none; picked: whether it has a list.
 */
ds_status ds_cache_attention_ex(const void* q, int32_t dtype, int64_t sequences, int32_t tokens, int32_t q_heads,
                                int32_t D, int64_t q_seq_stride, int64_t q_token_stride, int64_t q_head_stride,
                                const void* cache, const void* scales, int64_t pages, int32_t heads, int32_t page,
                                const int32_t* table, int64_t table_width, int64_t table_stride, const int32_t* lens,
                                const int32_t* indices, int32_t K, float scale, void* out, float* out_lse,
                                void* workspace, size_t workspace_bytes, cudaStream_t stream);
ds_status ds_cache_attention_workspace_bytes(int32_t dtype, int64_t sequences, int32_t tokens, int32_t q_heads, int32_t D,
                                             int32_t heads, int32_t page, int64_t table_width, int32_t picked, int32_t K,
                                             size_t* bytes);

/* ======================================================================================
 * What follows the selections: log probabilities of chosen tokens, the exchange of tokens with
 * their chosen experts, and the experts' products in 8 bits.  Rules as for the operators above.
 * ==================================================================================== */

/*
 * ds_token_logprobs -- per row x of V logits: lse = log sum exp(x), the given token's log
 * probability x_t - lse, the entropy -sum p log p of p = softmax(x), and the `top` largest
 * logits' tokens with their log probabilities, in descending order, equal logits by the lower
 * index (-0 equals +0).
 *   logits, dtype   row r starts at element r * row_stride (any stride >= V); -inf excludes a
 *                   token, whose log probability is -inf
 *   rows            0 .. 2^31 - 1;  1 <= V <= 2^30;  0 <= top <= min(V, 32)
 *   tokens          [rows] int32; outside [0, V): none is given, log probability 0
 *   out_logprobs, out_lse, out_entropy   [rows] floats
 *   out_top_logprobs, out_top_tokens     [rows, top] floats and int32 (unused with top = 0)
 * A row of -inf alone: lse and log probabilities -inf, entropy 0, its first tokens as the top.  A row with a NaN or
 * +inf: NaN for lse, entropy and all log probabilities (0 still where no token is given); its top lists NaN of either
 * sign before +inf.  Sums
 * are fp32, of exponentials off by 2^-22 of each; x is taken relative to the row's largest
 * before anything is rounded.
 */
ds_status ds_token_logprobs(const void* logits, int32_t dtype, int64_t rows, int64_t V, int64_t row_stride,
                            const int32_t* tokens, int32_t top, float* out_logprobs, float* out_lse, float* out_entropy,
                            float* out_top_logprobs, int32_t* out_top_tokens, cudaStream_t stream);

/*
 * ds_token_logprobs_backward -- the gradient of the given tokens' log probabilities and of the
 * entropies with respect to the logits:
 *   dx_v = g ([v = t] - p_v) - h p_v (log p_v + entropy),  p = exp(x - lse).
 *   grad_logprobs g [rows];  grad_entropy h [rows] or NULL (0)
 *   lse, entropy    as ds_token_logprobs gave them (entropy may be NULL where grad_entropy is)
 *   grad_logits     rows of V elements of dtype, row r at element r * grad_stride (>= V); every
 *                   element is written; must not overlap logits
 * A row without a given token has the entropy's part alone, a row of -inf alone zeros, a row whose lse is NaN
 * NaN throughout.  The top tokens'
 * log probabilities have no gradient here.  lse is rounded to fp32, which moves a row's p by at most 2^-19 of
 * themselves up to |lse| = 64; a row beyond is summed once more, so that p keeps its digits there too.
 */
ds_status ds_token_logprobs_backward(const float* grad_logprobs, const void* logits, int32_t dtype, int64_t rows,
                                     int64_t V, int64_t row_stride, const int32_t* tokens, const float* lse,
                                     const float* grad_entropy, const float* entropy, void* grad_logits,
                                     int64_t grad_stride, cudaStream_t stream);

/*
 * The experts' exchange.  Slot t * k + i is token t's i-th choice (ds_route's experts).
 *
 * ds_expert_sort ranks the slots by expert, equal experts by slot:
 *   experts   [tokens, k] int32; one outside [0, E) is no choice (a padded token's)
 *   places    [tokens, k] int32: the slot's rank, -1 for no choice
 *   offsets   [E + 1] int32: the first rank of each expert, then the number of choices
 * ds_expert_gather writes row t of x to row places[t, i] of out for each i, and zeros to the rows
 * of out ([tokens * k, D], dtype) behind the last choice.
 * ds_expert_combine: out[t] = sum_i weights[t, i] * y[places[t, i]], over the places in
 * [0, rows); sums in fp32, in order of i.  weights NULL: 1 (the gradient of ds_expert_gather).
 * ds_expert_combine_backward, for the gradient `grad` of out and y [tokens * k, D]:
 *   grad_y[places[t, i]] = weights[t, i] * grad[t] (rows behind the last choice: zeros),
 *   grad_weights[t, i] = grad[t] . y[places[t, i]] (0 for no choice); sums in fp32.
 * tokens >= 0, 1 <= k <= 32, tokens * k < 2^31, E <= 512, 1 <= D <= 2^30; x, y and grad take a row
 * stride >= D in elements, outputs are contiguous and overlap no input.  places and offsets are those of one
 * ds_expert_sort (places outside the rows are left out whatever they hold).
 */
ds_status ds_expert_sort(const int32_t* experts, int64_t tokens, int32_t k, int32_t E, int32_t* places,
                         int32_t* offsets, cudaStream_t stream);
ds_status ds_expert_gather(const void* x, int32_t dtype, int64_t tokens, int32_t D, int64_t row_stride,
                           const int32_t* places, int32_t k, const int32_t* offsets, int32_t E, void* out,
                           cudaStream_t stream);
ds_status ds_expert_combine(const void* y, int32_t dtype, int64_t rows, int32_t D, int64_t row_stride,
                            const int32_t* places, int64_t tokens, int32_t k, const float* weights, void* out,
                            cudaStream_t stream);
ds_status ds_expert_combine_backward(const void* grad, int64_t grad_stride, const void* y, int32_t dtype, int32_t D,
                                     int64_t row_stride, const int32_t* places, int64_t tokens, int32_t k,
                                     const int32_t* offsets, int32_t E, const float* weights, void* grad_y,
                                     float* grad_weights, cudaStream_t stream);

/*
 * The 8-bit form: codes of e4m3 and an fp32 scale for each block of 128 numbers of a row, or of
 * 128 x 128 numbers of a matrix; blocks at the edges are smaller.  A code c of a block with scale s
 * stands for c * s.
 *
 * ds_quantise_blocks: s is the least power of two >= 2^-126 with max |x| <= 448 s, c = e4m3(x / s),
 * rounded to nearest, ties to even (x / s is exact).  Infinities and NaN have the code NaN; for its block's scale
 * an infinity counts as fp32's largest number (s = 2^120), a NaN as 0.
 *   x, dtype    row r of matrix m at element m * matrix_stride + r * row_stride, K numbers
 *   block_rows  1 or 128
 *   codes       [matrices, rows, K] bytes;  scales [matrices, ceil(rows / block_rows),
 *               ceil(K / 128)] floats
 *   1 <= K <= 2^26
 * ds_expert_gather_quantised is ds_expert_gather with rows in that form: codes [tokens * k, D] bytes,
 * scales [tokens * k, ceil(D / 128)], D <= 2^26; rows behind the last choice are the form of zeros.
 */
ds_status ds_quantise_blocks(const void* x, int32_t dtype, int64_t matrices, int64_t rows, int32_t K,
                             int64_t matrix_stride, int64_t row_stride, int32_t block_rows, void* codes, float* scales,
                             cudaStream_t stream);
ds_status ds_expert_gather_quantised(const void* x, int32_t dtype, int64_t tokens, int32_t D, int64_t row_stride,
                                     const int32_t* places, int32_t k, const int32_t* offsets, int32_t E, void* codes,
                                     float* scales, cudaStream_t stream);

/*
 * ds_expert_product -- rows sorted by expert times each expert's weights, both in 8 bits:
 *   out[r, n] = sum_b x_scales[r, b] * w_scales[e, n / 128, b] * sum_{j in block b} x[r, j] w[e, n, j]
 * for the rows r in [offsets[e], offsets[e + 1]) of each expert e.  Products of codes are exact, a
 * block's are summed by the tensor cores and the blocks' sums in fp32.  Rows outside
 * [offsets[0], offsets[E]) are zeros.
 *   x           [rows, K] e4m3 codes, row r at byte r * x_stride;  x_scales [rows, ceil(K / 128)]
 *   w           [E, N, K] e4m3 codes, row n of expert e at byte e * w_matrix_stride + n *
 *               w_row_stride;  w_scales [E, ceil(N / 128), ceil(K / 128)], any fp32 scales
 *   offsets     [E + 1] int32, ascending, or NULL: one expert (E = 1) has all rows.  Others leave rows of out
 *               undefined; those outside [0, rows] count as its ends
 *   dtype, out  [rows, N] bf16 or fp32
 * K is a multiple of 16, x, w and their strides are 16-byte aligned, w_matrix_stride > 0 with several
 * experts; 0 <= rows <= 2^30, E <= 512, N and K <= 2^24.  Scales whose product leaves fp32's range
 * do not give finite numbers.  A wait inside the kernel that runs out (about a second) is recorded for
 * ds_get_device_status, and the outputs are then undefined.
 */
ds_status ds_expert_product(const void* x, const float* x_scales, int64_t rows, int32_t K, int64_t x_stride,
                            const void* w, const float* w_scales, int32_t E, int32_t N, int64_t w_row_stride,
                            int64_t w_matrix_stride, const int32_t* offsets, int32_t dtype, void* out,
                            cudaStream_t stream);

/* ds_expert_product in which every CTA gives its first tile up before that tile's block number `block` (>= 0) along
 * k, as if a wait had run out there: copies and products are in flight then.  The kernel records
 * DS_ERR_TIMEOUT for ds_get_device_status and returns, and out is undefined; tiles of no more blocks end as ever.
 * Checks the kernel's failure path without a GPU fault. */
ds_status ds_expert_product_probe(int32_t block, const void* x, const float* x_scales, int64_t rows, int32_t K,
                                  int64_t x_stride, const void* w, const float* w_scales, int32_t E, int32_t N,
                                  int64_t w_row_stride, int64_t w_matrix_stride, const int32_t* offsets, int32_t dtype,
                                  void* out, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DS_TOPK_H */
