/*
 * pkv.h -- C ABI of the GB300 (sm_103a) paged KV-cache hot path.
 *
 * The operations and names come from AstrAI's inference design
 * (docs/guides/inference.md):
 *   - "KV Cache": decode attention o_n = sum_j softmax(q_n k_j / sqrt(d_k)) v_j;
 *     RoPE is applied before the cache write;
 *   - "KVCache System": KVStorage k_buffer / v_buffer [n_layers, size,
 *     n_kv_heads, head_dim]; ReqToTokenPool req_to_token [num_reqs,
 *     max_ctx_len] (logical position -> physical token slot); the KVCache
 *     dataclass fields req_pool_indices, seq_lens, out_cache_loc, max_len,
 *     kv_indptr, qo_indptr; the write k_buffer[layer_id, out_cache_loc] = k;
 *   - "Attention Backend": decode writes K/V then attends through req_to_token
 *     with page_size 1; prefill writes K/V then attends over a ragged batch
 *     addressed by qo_indptr / kv_indptr;
 *   - "Rotary Embedding Backend": freqs_cis [max_len, dim/2, 2] f32 (cos, sin).
 * The commit log under tests/inference/test_cache.py fixes int32 page-table,
 * request-row and cache-location indices, and a workspace allocated once that
 * owns the split-K partials decode_o_part / decode_ml_part so that CUDA-graph
 * replay sees stable addresses.
 *
 * Conventions for every entry point:
 *   - All tensors are caller-owned, row-major and contiguous, in memory the
 *     GPU can address: device or managed memory, or registered (pinned)
 *     host memory mapped at the same address.  The pool, the index tables
 *     and the workspace belong in device memory; a step's small inputs and
 *     outputs (q, o, the new K/V rows, seq_lens, kv_indptr, qo_indptr,
 *     req_pool_indices, out_cache_loc) may stay in pinned host memory, which
 *     the kernels then read and write in place over the host link (on a
 *     Grace-Blackwell node: NVLink-C2C).  Any other address (unregistered
 *     host memory, say) returns PKV_ERR_ARG before anything is enqueued.
 *     The library never allocates, frees or copies host<->device.
 *   - `stream` is a cudaStream_t passed as void* (NULL: the legacy default
 *     stream).  Work is enqueued asynchronously; the call returns once enqueued.
 *   - Return value: PKV_OK or a negative PKV_ERR_* code.  Errors the host can
 *     see (null pointers, shapes, sizes, alignment, unsupported variants) are
 *     returned before anything is enqueued.  Errors in device-resident data
 *     (a slot outside [0, size), a request row outside [0, num_reqs), a length
 *     beyond max_ctx_len / max_len, kv_len < q_len) never fault: the kernel
 *     substitutes a safe index, records the first such error in a per-device
 *     error word and finishes; pkv_last_device_error() reports it.  Results
 *     of a call that recorded such an error are unspecified.
 *   - Nothing traps, aborts or waits without a bound.
 *   - The library looks up the device addresses of its own device-resident
 *     objects (the error word, the array of pkv_paged_decode_noalloc) once
 *     per device and keeps them for the life of the process.  After
 *     cudaDeviceReset() on a device those addresses are stale: make no
 *     further pkv_* call on that device in the same process.
 */
#ifndef PKV_H_
#define PKV_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Storage element type of k_buffer / v_buffer; q, k, v and o use the same. */
typedef enum { PKV_F32 = 0, PKV_BF16 = 1 } pkv_dtype;

enum {
    PKV_OK = 0,
    PKV_ERR_ARG = -1,         /* bad pointer, shape, size, alignment or index range */
    PKV_ERR_UNSUPPORTED = -2, /* valid request that this build has no kernel for */
    PKV_ERR_WORKSPACE = -3,   /* workspace missing, uninitialised or too small */
    PKV_ERR_INDEX = -4,       /* device data out of range (from pkv_last_device_error) */
    PKV_ERR_CUDA = -5         /* a CUDA runtime call or launch failed */
};

/*
 * The KVCache dataclass of "KVCache System", as plain pointers and sizes.
 *   k_buffer, v_buffer  [n_layers, size, n_kv_heads, head_dim] of dtype; the
 *                       row of (layer, slot) is n_kv_heads*head_dim elements.
 *   req_to_token        int32 [num_reqs, max_ctx_len]: physical slot of each
 *                       logical position of each request row.  page_size > 1
 *                       pools are expressed per token (a page is a run of
 *                       page_size consecutive slots).
 *   req_pool_indices    int32 [batch]: request row of each batch entry.
 *   seq_lens            int32 [batch]: decode context length of each entry,
 *                       INCLUDING the token written this step.
 *   kv_indptr           int32 [batch + 1]: prefix sums of the kv lengths
 *                       (kv_indptr[0] = 0); in prefill the kv length of entry b
 *                       is kv_indptr[b+1] - kv_indptr[b] (cached prefix + new
 *                       tokens).  In decode it is optional: when given, it
 *                       must equal the prefix sums of seq_lens, and the
 *                       automatic plan splits all tokens of the batch evenly
 *                       across the SMs (an entry whose differences disagree
 *                       with seq_lens is a device-data error).
 *   qo_indptr           int32 [batch + 1]: prefix sums of the query lengths
 *                       (prefill only; NULL in decode).
 *   out_cache_loc       int32 [n_new]: destination slot of each new token, in
 *                       qo_indptr order (the pages' [batch, seq_len] flattened).
 *   batch               number of batch entries.
 *   max_len             host-side upper bound of seq_lens (decode) or of the kv
 *                       lengths (prefill): the pages pass max(seq_lens) on the
 *                       host so that no device sync is needed.  Launch grids
 *                       are sized from it.
 */
typedef struct pkv_kvcache {
    void *k_buffer;
    void *v_buffer;
    int32_t dtype;            /* pkv_dtype */
    int32_t n_layers;
    int32_t n_kv_heads;
    int32_t head_dim;
    int64_t size;
    const int32_t *req_to_token;
    int32_t num_reqs;
    int32_t max_ctx_len;
    const int32_t *req_pool_indices;
    const int32_t *seq_lens;
    const int32_t *kv_indptr;
    const int32_t *qo_indptr;
    const int32_t *out_cache_loc;
    int32_t batch;
    int32_t max_len;
} pkv_kvcache;

/*
 * Caller-owned workspace for the decode split-K partials (the pages'
 * decode_o_part / decode_ml_part):
 *   o_part   float [max_batch, n_heads, max_splits, head_dim]: normalised
 *            attention output of each split of each (entry, head);
 *   ml_part  float [max_batch, n_heads, max_splits, 2]: (running max in base-2
 *            units of the scaled score, softmax denominator) of each split.
 * Allocate pkv_workspace_bytes(...) bytes of device memory once (256-byte
 * aligned, e.g. straight from cudaMalloc), describe it with
 * pkv_workspace_init(), and pass the same descriptor to every call so that
 * the device addresses stay fixed across CUDA-graph replays.  No call needs
 * its contents to persist between calls; calls that share a workspace must not
 * overlap on the GPU.
 */
typedef struct pkv_workspace {
    void *base;
    size_t bytes;
    int32_t max_batch;
    int32_t n_heads;
    int32_t head_dim;
    int32_t max_splits;
    float *o_part;
    float *ml_part;
    uint32_t magic;           /* set by pkv_workspace_init */
} pkv_workspace;

/* Bytes needed for a workspace of these dimensions (0 if any is < 1). */
size_t pkv_workspace_bytes(int32_t max_batch, int32_t n_heads, int32_t head_dim,
                           int32_t max_splits);

/* Fill *out to describe `base`.  PKV_ERR_ARG on null / misaligned base or bad
 * dimensions, PKV_ERR_WORKSPACE if `bytes` is smaller than required. */
int pkv_workspace_init(void *base, size_t bytes, int32_t max_batch, int32_t n_heads,
                       int32_t head_dim, int32_t max_splits, pkv_workspace *out);

/*
 * K/V cache write ("KVCache System": k_buffer[layer_id, out_cache_loc] = k):
 * for i in [0, n_new): row (layer_id, c->out_cache_loc[i]) of c->k_buffer
 * (resp. v_buffer) becomes k[i] (resp. v[i]).  k, v: [n_new, n_kv_heads,
 * head_dim] of c->dtype.  Bit-exact copy.  Requires 16-byte aligned buffers
 * and a row of n_kv_heads*head_dim elements that is a multiple of 16 bytes.
 * Duplicate destination slots give an unspecified one of the rows.  n_new = 0
 * is a no-op.  Reads c->out_cache_loc, c->size, c->n_layers, the buffers and
 * shape fields only.
 */
int pkv_kv_write(const pkv_kvcache *c, int32_t layer_id, const void *k, const void *v,
                 int32_t n_new, void *stream);

/*
 * Fused rotary embedding + K/V cache write ("KV Cache": RoPE before the
 * write; "Rotary Embedding Backend": freqs_cis [max_pos, head_dim/2, 2] f32).
 * Row i of k is rotated pairwise, (k[2e] + i k[2e+1]) * (cos + i sin) with
 * (cos, sin) = freqs_cis[positions[i], e], rounded once to the storage dtype,
 * and written like pkv_kv_write; v is copied unchanged.  positions: int32
 * [n_new] device array (a position outside [0, max_pos) is a device-data
 * error).  head_dim must be even.
 */
int pkv_rope_kv_write(const pkv_kvcache *c, int32_t layer_id, const void *k, const void *v,
                      int32_t n_new, const float *freqs_cis, int32_t max_pos,
                      const int32_t *positions, void *stream);

/*
 * Paged decode attention ("KV Cache" formula; "Attention Backend" decode path).
 * For each entry b < c->batch with request row r = c->req_pool_indices[b] and
 * context n = c->seq_lens[b], and each query head h < n_heads:
 *   o[b, h] = sum_{j<n} softmax_j(sm_scale * q[b,h] . K[slot_j, h/G]) V[slot_j, h/G],
 *   slot_j = c->req_to_token[r, j],  G = n_heads / c->n_kv_heads,
 * with K/V the rows of layer `layer_id`.  q, o: [batch, n_heads, head_dim] of
 * c->dtype; o must not alias q.  n = 0 gives o = 0.  Accumulation in fp32,
 * one rounding to the output dtype.  The work is split and the partials go
 * to the workspace, merged by a second kernel:
 *   - with c->kv_indptr (bf16, n_kv_heads in {1, 2, 4, 8}): the tokens of the
 *     whole batch, [0, kv_indptr[batch]), are divided evenly among up to one
 *     CTA per SM; the workspace must hold (CTAs + batch) x n_heads partial
 *     rows (else the chunked plan below is used);
 *   - otherwise each context is cut into chunks whose size is chosen on the
 *     host from c->max_len, c->batch and the SM count.
 * Without a workspace only single-split plans are possible.
 * Supported: head_dim 64 or 128, G in {1, 2, 4, 8}.
 */
int pkv_paged_decode(const pkv_kvcache *c, int32_t layer_id, const void *q, void *o,
                     int32_t n_heads, float sm_scale, const pkv_workspace *ws, void *stream);

/*
 * pkv_paged_decode with a shared prefix stated: the first shared_len
 * positions of every request row of the batch (req_to_token[r, 0 ..
 * shared_len), r = c->req_pool_indices[b]) hold the same slots, as when the
 * prefix cache ("KVCache System") hands several tasks the same pages.  Same
 * operation and result as pkv_paged_decode; with the balanced plan, 8 kv
 * heads, shared_len >= 64, batch >= 2 and room in the workspace the shared
 * rows are read once per launch at head_dim 128 and once per group of 16 / G
 * requests at head_dim 64 (see pkv_paged_decode_pages for how, and for the
 * workspace it needs), otherwise the statement is ignored.  Every seq_len
 * must be >= shared_len; a shorter context, or a row whose leading slots
 * differ from the first entry's (head_dim 128) or its group's (head_dim
 * 64), is a device-data error.  shared_len < 0, or shared_len > c->max_len,
 * returns PKV_ERR_ARG.
 */
int pkv_paged_decode_shared(const pkv_kvcache *c, int32_t layer_id, int32_t shared_len,
                            const void *q, void *o, int32_t n_heads, float sm_scale,
                            const pkv_workspace *ws, void *stream);

/*
 * Paged decode through a page table ("KVCache System": the pool is made of
 * pages of page_size consecutive token slots; the 5-D view [n_layers,
 * n_pages, page_size, n_kv_heads, head_dim] is byte-identical to
 * c->k_buffer's [n_layers, size, n_kv_heads, head_dim] with size = n_pages *
 * page_size).  Position j of entry b reads slot
 *   req_to_page[r * max_pages + j / page_size] * page_size + j % page_size,
 * r = c->req_pool_indices[b]; a 16-token stage of the kernel is then a run of
 * consecutive slots.  req_to_page: int32 [c->num_reqs, max_pages] device
 * array (c->num_reqs is its row count); c->req_to_token and c->max_ctx_len
 * are not read.  Otherwise the operation, arguments, results and plan are
 * those of pkv_paged_decode, with c->max_len <= max_pages * page_size.
 * Requires c->size to be a multiple of page_size.  Supported: bf16,
 * head_dim 64 or 128, G and n_kv_heads in {1, 2, 4, 8}.  A page index
 * outside [0, size / page_size) is a device-data error.
 *
 * shared_pages: the caller's statement that the first shared_pages pages of
 * every row of the batch are the same pages (a prefix shared by all
 * requests, "KVCache System" prefix cache hits); 0 states nothing.  It does
 * not change the result: with 8 kv heads, at least 64 shared positions
 * (Ts = shared_pages * page_size), batch >= 2 and room in the workspace it
 * lets the decode read each shared K/V row fewer times than once per
 * request, and merge the two parts; otherwise it is ignored.
 *   - head_dim 128: once per launch.  A tensor-core kernel attends all
 *     batch x G query heads of each kv head to the prefix (read from the
 *     first entry's row) in chunks of at most 512 positions, one CTA per
 *     (chunk, kv head, 256 query rows), while the split kernel takes every
 *     entry's positions past the prefix on the other SMs.  The workspace
 *     then holds (CTAs + batch) x n_heads rows plus ceil(Ts / 512) x batch x
 *     n_heads more, CTAs being the SM count minus the tensor-core kernel's.
 *   - head_dim 64: once per group of 16 / G consecutive requests, inside the
 *     split kernel; the workspace holds (CTAs + batch) x n_heads rows plus
 *     (CTAs + ceil(batch / (16 / G))) x (16 / G) x n_heads more.
 * Every seq_len must be >= Ts; a shorter context, or a row whose leading
 * pages differ from the first entry's (head_dim 128) or its group's
 * (head_dim 64), is a device-data error.  shared_pages < 0, or shared
 * positions beyond c->max_len, returns PKV_ERR_ARG.
 */
int pkv_paged_decode_pages(const pkv_kvcache *c, int32_t layer_id, const int32_t *req_to_page,
                           int32_t max_pages, int32_t page_size, int32_t shared_pages,
                           const void *q, void *o, int32_t n_heads, float sm_scale,
                           const pkv_workspace *ws, void *stream);

/*
 * One decode step of a layer ("Attention Backend": the new tokens' K/V go
 * into the cache, then attention reads it): pkv_kv_write of k_new / v_new
 * (n_new rows at c->out_cache_loc, n_new may be 0) followed by
 * pkv_paged_decode with the automatic plan.  Arguments, layouts, results and
 * errors are those of the two calls made back to back on `stream`; both are
 * validated before either is enqueued.  The tensor-core decode kernel is
 * launched as a programmatic dependent of the write: it reads kv_indptr,
 * req_pool_indices, seq_lens, req_to_token and q while the write runs and
 * waits for the write before reading K/V rows.  Those inputs therefore follow
 * plain stream order (the write never modifies them).  When q (bf16) is in
 * pinned host memory and the workspace has room past the partial rows the
 * call uses, the write also copies q into that room once, and the decode
 * reads the copy after its wait instead of q over the host link; the result
 * is the same either way.
 */
int pkv_decode_step(const pkv_kvcache *c, int32_t layer_id, const void *k_new, const void *v_new,
                    int32_t n_new, const void *q, void *o, int32_t n_heads, float sm_scale,
                    const pkv_workspace *ws, void *stream);

/*
 * pkv_paged_decode with an explicit split size: every entry's context is cut
 * into chunks of `chunk` tokens (a positive multiple of 32; 0 = automatic).
 * The result is the same up to fp32 rounding for any chunk; the workspace
 * must hold ceil(c->max_len / chunk) splits.
 */
int pkv_paged_decode_chunked(const pkv_kvcache *c, int32_t layer_id, const void *q, void *o,
                             int32_t n_heads, float sm_scale, int32_t chunk,
                             const pkv_workspace *ws, void *stream);

/*
 * The plan pkv_paged_decode would use: *chunk tokens per split and
 * *n_splits = ceil(c->max_len / *chunk) splits, or *chunk = 0 and *n_splits =
 * the number of CTAs when the tokens are divided evenly over kv_indptr.
 * Host-only; enqueues nothing.
 */
int pkv_decode_plan(const pkv_kvcache *c, int32_t n_heads, const pkv_workspace *ws,
                    int32_t *chunk, int32_t *n_splits);

/*
 * Ragged paged prefill ("Attention Backend" prefill path).  Entry b has
 * q_len = qo_indptr[b+1] - qo_indptr[b] new tokens (already written to the
 * cache) at the end of a context of kv_len = kv_indptr[b+1] - kv_indptr[b]
 * positions, so its cached prefix is P = kv_len - q_len.  Packed query row
 * p = qo_indptr[b] + i, head h attends over positions j < P + i + 1 when
 * `causal` (the mask of process_attention_mask: a cached prefix is fully
 * visible), else j < kv_len, reading slot req_to_token[req_pool_indices[b], j]
 * of kv head h / G.  q, o: [qo_indptr[batch], n_heads, head_dim] bf16.
 * max_q_len / max_kv_len: host-side upper bounds of q_len and kv_len (grid
 * sizing; max_q_len * G at most 65535 * 256 rows, else PKV_ERR_ARG).  The
 * CTAs launch the kv heads of a query-tile pair together, the pairs of an
 * entry longest first, then the entries.  An entry whose rows [qo_indptr[b], qo_indptr[b+1]) do not lie
 * within [0, qo_indptr[batch]), or whose lengths break these bounds, is a
 * device-data error: its rows of q and o are neither read nor written.
 * `ws` may be NULL.  With a workspace (pkv_workspace_init; its o_part must
 * hold 8 ints per entry) and 2 to 256 entries, a one-CTA planning kernel
 * checks the entries and ranks them by decreasing kv_len into the start of
 * o_part, and the prefill, launched as its programmatic dependent, takes the
 * entries in that order: the longest start first and the short ones fill
 * the SMs at the end.  The result is the same bits in either order.  The
 * workspace serves one call at a time (as for the decode).  Supported: bf16,
 * head_dim 64 or 128 (5th-generation tensor cores, accumulators in tensor
 * memory), G in {1, 2, 4, 8}.
 */
int pkv_paged_prefill(const pkv_kvcache *c, int32_t layer_id, const void *q, void *o,
                      int32_t n_heads, int32_t max_q_len, int32_t max_kv_len, int32_t causal,
                      float sm_scale, const pkv_workspace *ws, void *stream);

/*
 * Tables of a step, built on the GPU ("KVCache System": the page table, the
 * slot maps and the prefix sums that the host otherwise computes from the
 * requests' lengths).  Entry b < c->batch has context length n =
 * c->seq_lens[b] INCLUDING its q = q_lens[b] new tokens (q_lens NULL: one new
 * token for each entry with n > 0), which stand at positions [n - q, n) of
 * request row r = c->req_pool_indices[b].  With ps = page_size:
 *   - its pages ceil((n-q)/ps) .. ceil(n/ps)-1 are new: the entries take
 *     them in entry order from free_pages[*free_start ..], lowest page of the
 *     entry first, and they are written to req_to_page[r];
 *   - *free_end = *free_start + the pages taken.  The two are different words
 *     (a step that is replayed from a CUDA graph swaps or copies them);
 *   - kv_indptr[b+1] and qo_indptr[b+1] (each may be NULL) are the prefix sums
 *     of n and q, [0] = 0;
 *   - new token i, in entry order (the order of qo_indptr), gets positions[i]
 *     (may be NULL), out_cache_loc[i] = page * ps + position % ps with the
 *     page of req_to_page, and, where req_to_token is given,
 *     req_to_token[r, position] = the same slot.
 * All arrays are int32 device arrays.  out_cache_loc and positions hold
 * max_new entries (2^30 at most); what lies behind the last new token is left as it was, and
 * so are table columns of positions that are not new.  The pages of earlier
 * positions (a partly filled last page, a cached prefix) are read from
 * req_to_page.  One kernel; nothing is allocated.
 * Reads c->batch, c->req_pool_indices, c->seq_lens, c->num_reqs,
 * c->max_ctx_len (with req_to_token) and c->size (a multiple of page_size).
 * Request rows of entries with new tokens must be distinct within a call
 * (else the tables of a row that stands twice are unspecified).
 * Device-data errors: a request row outside [0, num_reqs), n outside
 * [0, max_pages * ps] (or beyond max_ctx_len with req_to_token), q outside
 * [0, n] (such an entry counts as n = q = 0); more new tokens than max_new
 * (those beyond get no slot; the pages of all are taken and entered in
 * req_to_page); a prefix sum beyond 2^31 - 1; a page outside
 * [0, size / ps) in req_to_page or free_pages, or a free list that runs out
 * (the tokens concerned get slot -1, and new pages of theirs -1, which the
 * write refuses in turn); *free_start outside [0, n_free].
 */
typedef struct pkv_tables {
    const int32_t *q_lens;       /* [batch], or NULL */
    int32_t *req_to_page;        /* [num_reqs, max_pages], in and out */
    int32_t max_pages;
    int32_t page_size;
    const int32_t *free_pages;   /* [n_free] */
    const int32_t *free_start;   /* [1] */
    int32_t *free_end;           /* [1] */
    int32_t n_free;
    int32_t max_new;
    int32_t *kv_indptr;          /* [batch + 1], or NULL */
    int32_t *qo_indptr;          /* [batch + 1], or NULL */
    int32_t *positions;          /* [max_new], or NULL */
    int32_t *out_cache_loc;      /* [max_new] */
    int32_t *req_to_token;       /* [num_reqs, max_ctx_len], or NULL */
} pkv_tables;

int pkv_build_tables(const pkv_kvcache *c, const pkv_tables *t, void *stream);

/*
 * Sparse decode: attention over the pages that a cheap score selects for each
 * query.  The cache is a pool of pages of page_size consecutive slots behind a
 * page table (as for pkv_paged_decode_pages; c->req_to_token and
 * c->max_ctx_len are not read), and beside the pool stands, for each page and
 * kv head, the channelwise minimum and maximum of the keys written to it:
 *   page_bounds  [n_layers, size / page_size, n_kv_heads, 2, head_dim] of
 *                c->dtype, minimum at [.., 0, :], maximum at [.., 1, :];
 *   req_to_page  int32 [num_reqs, max_pages];
 *   top_k        pages selected per (entry, kv head) at most; n_first and
 *                n_last of them are the context's first and last pages
 *                (n_first + n_last <= top_k).
 * An entry of c->req_pool_indices / c->seq_lens is one query.  The queries of
 * a prompt, or of a speculative draft, are entries that name the same request
 * row with growing seq_lens.
 */
typedef struct pkv_pages {
    void *page_bounds;
    const int32_t *req_to_page;
    int32_t max_pages;
    int32_t page_size;
    int32_t top_k;
    int32_t n_first;
    int32_t n_last;
} pkv_pages;

/*
 * Bring page_bounds of layer `layer_id` up to date with the n_new keys that
 * were written to the slots c->out_cache_loc[0 .. n_new) of c->k_buffer (by
 * pkv_kv_write, pkv_rope_kv_write or pkv_decode_step on the same stream).
 * A key at the first slot of a page starts the page's bounds anew; other keys
 * widen the bounds that the page has.  The new tokens of a page stand next to
 * each other in out_cache_loc in ascending slot order, with or without gaps, as
 * pkv_build_tables and the prefill's order give them (else that page's bounds
 * are unspecified).  Exact; a NaN key makes its channel's bounds NaN.  Requires
 * 16-byte aligned page_bounds and head rows of a multiple of 16 bytes.  Slots
 * outside [0, size) are device-data errors and are passed over.  n_new = 0 is a
 * no-op.  Does not read req_to_page.
 */
int pkv_page_bounds(const pkv_kvcache *c, int32_t layer_id, const pkv_pages *pg, int32_t n_new,
                    void *stream);

/*
 * Select pages.  For entry b with N = ceil(c->seq_lens[b] / page_size) pages,
 * kv head g and page p:
 *   score = max over the G query heads h of the group of
 *           sum_c max(q[b,h,c] * minimum[c], q[b,h,c] * maximum[c]),
 * the largest product that the query can have with any key inside the page's
 * bounds (those of every key written to the page, also behind the query's own
 * context).  With N <= top_k every page is selected; otherwise the first n_first
 * and the last n_last pages, and of the rest the top_k - n_first - n_last of
 * largest score.  The order is that of the scores in 64 bits: scores are
 * computed in 32 bits with a bound on their error, and those that the bound
 * leaves undecided are computed again in 64.  Equal scores go to the lowest
 * page, NaN ranks above every number.
 *   sel         int32 [batch, n_kv_heads, top_k]: logical pages, ascending,
 *               then -1;
 *   sel_counts  int32 [batch, n_kv_heads]: min(N, top_k).
 * A context whose length is 0 gets the count 0.  q: [batch, n_heads,
 * head_dim] of c->dtype.  Scores go to the workspace, which serves one call at
 * a time: ws->bytes must be
 * pkv_select_workspace_bytes(...) at least (ws may be NULL while c->max_len
 * needs no more than top_k pages).  A context has 2^30 pages at most.
 * Supported: f32 and bf16, head_dim 64 or
 * 128, G in {1, 2, 4, 8}.  A request row outside [0, num_reqs) (count 0), a
 * length outside [0, c->max_len] (clamped) and a page outside [0, size /
 * page_size) (page 0 in its place) are device-data errors.
 */
int pkv_select_pages(const pkv_kvcache *c, int32_t layer_id, const pkv_pages *pg, const void *q,
                     int32_t n_heads, int32_t *sel, int32_t *sel_counts, const pkv_workspace *ws,
                     void *stream);

/* Workspace bytes that pkv_select_pages needs (0 if any argument is < 1). */
size_t pkv_select_workspace_bytes(int32_t batch, int32_t n_kv_heads, int32_t max_len,
                                  int32_t page_size);

/*
 * Paged decode attention over selected pages: pkv_paged_decode_pages with the
 * sum of entry b, kv head g running over the positions j < c->seq_lens[b] that
 * lie in the logical pages sel[b, g, 0 .. sel_counts[b, g]) only.  sel:
 * int32 [batch, n_kv_heads, pg->top_k] (any order; a page that is listed twice
 * counts twice), sel_counts: int32 [batch, n_kv_heads].  No selected position
 * gives o = 0.  Reads neither page_bounds nor n_first / n_last and needs no
 * workspace: the CTAs that share an entry's kv head form a thread-block
 * cluster and join their partials in shared memory.  Accumulation in fp32, one
 * rounding to the output dtype.  A selected value that is not finite makes its
 * channel of its group's outputs not finite.  Supported: f32 and bf16, head_dim
 * 64 or 128, G in {1, 2, 4, 8}, 65535 kv heads at most (32767 for f32 with G =
 * 8).  Device-data errors as for pkv_select_pages, and a count
 * outside [0, top_k] (clamped) or a listed page outside the context (skipped).
 */
int pkv_paged_decode_selected(const pkv_kvcache *c, int32_t layer_id, const pkv_pages *pg,
                              const int32_t *sel, const int32_t *sel_counts, const void *q, void *o,
                              int32_t n_heads, float sm_scale, void *stream);

/*
 * One sparse decode step of a layer: pkv_kv_write of k_new / v_new (n_new rows
 * at c->out_cache_loc, n_new may be 0), pkv_page_bounds, pkv_select_pages and
 * pkv_paged_decode_selected, made back to back on `stream` with the later
 * launches overlapping the earlier ones.  Arguments, results and errors are
 * those of the four calls; all are validated before any is enqueued.
 */
int pkv_sparse_decode_step(const pkv_kvcache *c, int32_t layer_id, const pkv_pages *pg,
                           const void *k_new, const void *v_new, int32_t n_new, const void *q,
                           void *o, int32_t n_heads, float sm_scale, int32_t *sel,
                           int32_t *sel_counts, const pkv_workspace *ws, void *stream);

/*
 * The life of a cache's pages on the GPU.  pkv_build_tables takes pages from a
 * free list; the calls below share, copy, give back and move them.  They work
 * on the page table of pkv_build_tables and on one more array:
 *   shares      int32 [size / page_size]: references to each page beyond the
 *               first, never below 0 between calls.  0 for a free page and for one that a single request
 *               row holds, so that the pages of pkv_build_tables need no entry;
 *               a caller that holds a page by other means than the table (a
 *               cached prefix) adds one for it.
 *   free_pages  int32 [n_free], free_start, free_end: as for
 *               pkv_build_tables.  Taking pages moves the list's place
 *               forward, giving back moves it backward and writes the pages in
 *               front of it.
 *   req_to_token (may be NULL) [num_reqs, c->max_ctx_len] and page_bounds (may
 *               be NULL) are kept in step where they are given.
 * None of the calls allocates or waits.  A page that several rows hold is not
 * to be written to: before a row writes into a shared page (its length was cut
 * back into one), give it a page of its own (pkv_copy_pages).
 */
typedef struct pkv_page_state {
    int32_t *req_to_page;        /* [num_reqs, max_pages], in and out */
    int32_t max_pages;
    int32_t page_size;
    int32_t *shares;             /* [size / page_size], in and out */
    int32_t *free_pages;         /* [n_free] */
    const int32_t *free_start;   /* [1] */
    int32_t *free_end;           /* [1], not free_start's word */
    int32_t n_free;
    int32_t *req_to_token;       /* [num_reqs, max_ctx_len], or NULL */
    void *page_bounds;           /* [n_layers, size / page_size, n_kv_heads, 2, head_dim], or NULL */
} pkv_page_state;

/*
 * For i < n: page dst[i] becomes a copy of page src[i], in k_buffer, v_buffer
 * and page_bounds (where given) of every layer.  Bit-exact.  src, dst: int32
 * [n] device arrays; a pair whose src is -1, or whose two pages are the same,
 * is passed over.  A page may be the source of several pairs; a page that is
 * the destination of two pairs, or of one and the source of another, ends
 * with unspecified contents.  Other pages outside [0, size / page_size) are
 * device-data errors, and their pairs are passed over.  Requires 16-byte
 * aligned buffers (page_bounds too) and, as the calls below that copy, less
 * than 2^30 16-byte chunks in a page's rows and bounds of all layers.
 */
int pkv_copy_pages(const pkv_kvcache *c, int32_t page_size, void *page_bounds, const int32_t *src,
                   const int32_t *dst, int32_t n, void *stream);

/*
 * Fork request rows.  For entry b < c->batch the row r = c->req_pool_indices[b]
 * takes over the first n = c->seq_lens[b] positions of row parents[b] (int32
 * [batch]).  With ps = page_size:
 *   - the pages of its floor(n / ps) full pages are the parent's, and their
 *     shares go up by one;
 *   - a partly filled last page is a page of its own: the entries take one each
 *     from free_pages[*free_start ..] in entry order, and the parent page's
 *     first n % ps rows of every layer, and its bounds (those of all keys
 *     written to the parent's page), are copied to it;
 *   - *free_end = *free_start + the pages taken;
 *   - req_to_token[r, 0 .. n) is written where it is given.
 * What the row held before is forgotten (pkv_release_pages gives it back).
 * A parent may have several children in one call; the rows that take over must
 * be distinct and no entry's parent (else the tables, counts and copied pages
 * of the rows concerned are unspecified).  Device-data errors: a row outside
 * [0, num_reqs), a row forked from itself, a length outside [0, max_pages * ps]
 * (or beyond max_ctx_len with req_to_token) - such an entry counts as n = 0 -;
 * a page of the parent outside [0, size / ps) (-1 in its place; where it is the
 * partly filled one, the row has its page of the free list, without the copy);
 * a free list that runs out (-1), or holds such a page; *free_start outside [0,
 * n_free] (the list counts as empty).
 */
int pkv_fork_requests(const pkv_kvcache *c, const pkv_page_state *t, const int32_t *parents,
                      void *stream);

/*
 * Give pages back.  Entry b < c->batch keeps the first keep_lens[b] (int32
 * [batch]; NULL: 0) of the n = c->seq_lens[b] positions of row
 * c->req_pool_indices[b]: its pages ceil(keep / ps) .. ceil(n / ps) - 1 lose
 * one reference each and their entries of req_to_page become -1.  A page whose
 * last reference that was is free: the m pages that this call frees are
 * written to free_pages[*free_start - m .. *free_start) in ascending order,
 * and *free_end = *free_start - m.  The order does not depend on that of the
 * entries.  Reads neither the pool's rows nor c->max_len; req_to_token and
 * page_bounds are left as they are.  Device-data errors: a row outside [0,
 * num_reqs), a length outside [0, max_pages * ps], keep outside [0, n] (such
 * an entry gives nothing back); a table entry outside [0, size / ps) (passed
 * over; of a row that is named twice the second finds -1); more references
 * dropped than a page has (the page is freed once); m above *free_start (the
 * lowest pages are lost, and *free_end is 0); *free_start outside [0, n_free].
 */
int pkv_release_pages(const pkv_kvcache *c, const pkv_page_state *t, const int32_t *keep_lens,
                      void *stream);

/*
 * Move the used pages to the pool's front.  A page is free if it stands in
 * free_pages[*free_start .. n_free), used if not; U pages are used.  The used
 * pages behind the first U go to the free pages among the first U, lowest to
 * lowest, with their rows of every layer, their bounds and their shares.  Then
 *   remap       int32 [size / page_size]: where each page went; itself for
 *               pages that stay and for free ones;
 *   req_to_page, req_to_token (where given): every entry in range, of all
 *               num_reqs rows, follows remap; others stay as they are;
 *   free_out    int32 [n_free]: free_out[*free_start ..] = U, U + 1, ...;
 *               what lies before is not written.  May be free_pages itself.
 * The list's place stays where it is; free_end is not used.  The workspace
 * (pkv_compact_workspace_bytes) serves one call at a time.  Device-data
 * errors: a page in the list outside [0, size / page_size), or a second time
 * (the free pages are the others, and as many places at free_out's end are -1);
 * *free_start outside [0, n_free] (no page counts as free).
 */
int pkv_compact_pages(const pkv_kvcache *c, const pkv_page_state *t, int32_t *free_out,
                      int32_t *remap, const pkv_workspace *ws, void *stream);

/* Workspace bytes that pkv_compact_pages needs (0 if n_pages < 1). */
size_t pkv_compact_workspace_bytes(int64_t n_pages);

/*
 * Attention of a chunk of new tokens through the page table of
 * pkv_paged_decode_pages: drafts to verify, the next part of a prompt, single
 * tokens beside both, or (causal = 0) queries over the states of an encoder.
 * Entry b has the q_len = qo_indptr[b+1] - qo_indptr[b] rows from qo_indptr[b]
 * on of q and o, and a context of n = c->seq_lens[b] positions.  Its row i,
 * head h attends over the positions j <= n - q_len + i (causal: its new tokens,
 * already written to the cache, are the last of the context) or over all n;
 * position j is slot req_to_page[r * max_pages + j / page_size] * page_size +
 * j % page_size, r = c->req_pool_indices[b].  A row that sees no position (n =
 * 0; causal and n < q_len: the first q_len - n rows) gives 0.  q_len and n need
 * not agree otherwise.  What a row does not see has no part in its result,
 * whatever values stand there.  A value that a row sees and that is not finite
 * makes its channel of that row's outputs not finite; a score that is NaN or
 * +inf, or scores that are all -inf, make them NaN.
 *   q, o        [n_q, n_heads, head_dim] of c->dtype, o not q; rows of o that
 *               belong to no entry are left as they are.
 *   max_q_len   host-side bound of q_len (max_q_len * G at most 65535 * 64);
 *   c->max_len  that of n, max_pages * page_size and 2^30 at most.
 * The rows of two entries must not be the same (else they hold either's result).
 * Entries of one or a few rows beside one of thousands are right, but each is then
 * read by one CTA per kv head: a call of their own takes them faster.
 * Scores, sums and outputs are held in fp32 and rounded once to the output;
 * bf16 rounds the softmax's weights to bf16 for their product with V.  With few
 * query rows the contexts are cut into pieces whose partials go to the
 * workspace and are joined by a second kernel.  A workspace of
 * pkv_chunk_workspace_bytes(...) holds them; with less (ws->bytes), or none, the
 * contexts stay whole (or, fp32 and bf16 of more than 128 rows per entry, in
 * fewer pieces): the same result up to fp32 rounding, later.  The workspace
 * serves one call at a time.  Reads c->seq_lens, c->qo_indptr,
 * c->req_pool_indices, c->num_reqs and the pool; not c->req_to_token,
 * c->kv_indptr.  Supported: f32 and bf16, head_dim 64 or 128, G in {1, 2, 4, 8}.
 * Device-data errors: a request row outside [0, num_reqs), rows outside [0,
 * n_q), q_len outside [0, max_q_len], n outside [0, c->max_len] (the entry's
 * rows are neither read nor written); a page outside [0, size / page_size)
 * (page 0 in its place).
 */
int pkv_paged_chunk(const pkv_kvcache *c, int32_t layer_id, const int32_t *req_to_page,
                    int32_t max_pages, int32_t page_size, const void *q, void *o, int32_t n_q,
                    int32_t n_heads, int32_t max_q_len, int32_t causal, float sm_scale,
                    const pkv_workspace *ws, void *stream);

/* Workspace bytes of a pkv_paged_chunk call of these sizes (c->batch, c->max_len,
 * the pool's heads and types; n_q rows of q), 256 at least; 0 for sizes that it
 * refuses.  A call of fewer rows or a smaller batch may use more than one of the
 * largest: size it for each, or take what fits. */
size_t pkv_chunk_workspace_bytes(const pkv_kvcache *c, int32_t n_q, int32_t n_heads,
                                 int32_t max_q_len);

/*
 * Paged decode for callers that cannot allocate device memory: code running
 * while another component holds a stream capture open in global mode (where
 * cudaMalloc is not allowed), plugins inside engines whose allocator owns all
 * device memory, or latency-bound loops that cannot take cudaMalloc's
 * implicit synchronisation.  The pages have no counterpart: their decode always
 * receives a workspace.
 *
 * Same operation, arguments and results as pkv_paged_decode, but the split-K
 * partials live in a library-owned device array of 8 MiB (a file-scope
 * __device__ object that every GPU loading the library holds until the
 * process exits).  Nothing is allocated or freed.  The number of splits is
 * capped by what fits in the array for batch x n_heads x head_dim.  When not
 * even one split per (entry, head) fits, contexts of up to 2048 tokens
 * (c->max_len <= 2048) are decoded in one split with o written directly;
 * longer ones, or contexts that would need chunks over 2048 tokens, return
 * PKV_ERR_WORKSPACE.
 * The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current; make that first call
 * before any stream capture.  Every call on a device shares the one array
 * and leaves its partials there (nothing in it has to start at zero): calls
 * that overlap on the GPU, on any streams, race and give wrong results.
 */
int pkv_paged_decode_noalloc(const pkv_kvcache *c, int32_t layer_id, const void *q, void *o,
                             int32_t n_heads, float sm_scale, void *stream);

/*
 * Synchronise `stream`, then read and clear the calling device's error word.
 * Returns PKV_OK, PKV_ERR_INDEX (an error recorded on the device since the
 * last read) or PKV_ERR_CUDA.  *detail, if non-NULL, receives the first
 * recorded value: the offending slot, page, request row, length or position
 * itself, or one of these codes:
 *   -1000 - k      a decode wait on the copies of stage k gave up;
 *   -2001, -2007   a prefill wait gave up (producer, softmax warps);
 *   -3002 .. -3006 a prefill wait of the thread issuing tensor-core
 *                  instructions gave up;
 *   -5001 .. -5003, -5008 .. -5011
 *                  a wait of pkv_paged_chunk (bf16, more than 128 rows of
 *                  position and head in group per entry) gave up: copies of K,
 *                  of V, products, the look at V, the softmax;
 *   -5101 .. -5105 the same with up to 128 rows: copies, products, query
 *                  tiles, the look at V, the softmax.  After one of these
 *                  codes that call's outputs are unspecified;
 *   -100000 - b    a shared prefix was stated, but entry b's leading pages (or
 *                  slots) differ from the first entry's (head_dim 128) or
 *                  from its group's first entry's (head_dim 64);
 *   -200000 - c    shared-prefix CTA c was handed more positions than it
 *                  stages (not expected: the host sizes the grid for it);
 *   -300000 - b    the free list of pkv_build_tables or pkv_fork_requests ran
 *                  out at entry b;
 *   -400000 - p    pkv_release_pages dropped more references to page p than
 *                  there were.
 * An offending value can itself be negative (a negative slot, say).
 */
int pkv_last_device_error(void *stream, int64_t *detail);

/* Static, human-readable text for a status code. */
const char *pkv_status_string(int status);

/* Library version string. */
const char *pkv_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H_ */
