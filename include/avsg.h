/*
 * avsg.h -- C interface of the GB300 sparse-KV reuse decode step.
 *
 * The operation (AVSG page, arxivdaily 2609.37538, English abstract): dynamic
 * sparse attention selects, per decode step, a subset of token ids of each
 * (request, kv-head); the full KV cache lives in host memory.  This library
 * keeps a device (HBM) buffer of B slots per (request, kv-head) *unit* and, on
 * every step,
 *   1. matches the selected ids against the ids resident in the buffer,
 *   2. reserves victim slots for the ids that are not resident (bucketed LRU,
 *      Spin page "Unifying Sparse Attention with Hierarchical Memory for
 *      Scalable Long-Context LLM Serving", section 2B),
 *   3. copies only those missing KV rows from host memory into their slots,
 *      spreading the copy evenly over the GPU's SMs,
 *   4. runs decode attention of every query head over the selected rows.
 * Multi-token prediction: with n_tok > 1 query tokens per step, one shared
 * reservation covers the union of the tokens' selections (same abstract).
 *
 * Within a step the copy of the misses (bound by the host link) overlaps the
 * reservation and the attention over the selected rows that were already
 * resident: the library runs the gather (into a staging area), the
 * reservation, the hash-table update and the move of the previous step's
 * staged rows into their slots on three internal streams, forked from and
 * joined back into the caller's stream with events.  A step's missed rows
 * reach their slots during the next step (its hits on them read the staged
 * copy); avsg_read_state, avsg_set_budget and avsg_clear_error move them
 * first, so every entry point sees the buffer of the step-by-step order.
 *
 * Reservation order (the pages give no formula; this is the reading the
 * library implements): empty slots first, by ascending slot index; then the
 * slots not selected in this step, by bucket min(63, t - last_step) from 63
 * down to 1, ties by ascending slot index.  The i-th missing id in ascending
 * id order takes the i-th reserved slot.  Every selected id ends the step
 * with last_step = t.  The outcome is deterministic: slot maps, hit flags,
 * tags and buffer rows are identical run to run.
 *
 * Threading: a handle is used by one host thread and one CUDA stream at a
 * time.  All device work of a step is enqueued on the caller's stream with no
 * host synchronisation; avsg_get_stats and avsg_read_state synchronise.
 */
#ifndef AVSG_H_
#define AVSG_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define AVSG_VERSION 1

/* Return codes.  0 is success; every error is negative. */
#define AVSG_OK 0
#define AVSG_ERR_INVALID_ARG (-1)   /* null pointer, bad size or bad config field */
#define AVSG_ERR_CAPACITY (-2)      /* n_tok * k exceeds the buffer slots, or k > max_select */
#define AVSG_ERR_CUDA (-3)          /* a CUDA runtime call failed; see avsg_cuda_error */
#define AVSG_ERR_BAD_SELECTION (-4) /* device: id outside [0, num_entries), or repeated in one token */
#define AVSG_ERR_TIMEOUT (-5)       /* device: a bounded wait gave up */
#define AVSG_ERR_BAD_STEP (-6)      /* t is negative or not larger than the previous step's t */
#define AVSG_ERR_UNSUPPORTED (-7)   /* shape without a compiled attention kernel */
#define AVSG_ERR_LATCHED (-8)       /* a device error is pending; call avsg_clear_error */
#define AVSG_ERR_INTERNAL (-9)      /* device: an index check of the bounds-checked build failed */

/* avsg_config.flags */
#define AVSG_FLAG_NO_REUSE 1u /* no buffer reuse: copy every selected row every step */
/* The miss gather is assigned by request: one CTA copies all the misses of one
 * request (its kv-heads' units), the assignment the AVSG page measures its even
 * split against.  Default: the misses of all units are split evenly over the
 * gather's CTAs.  Results are identical either way; only the copy's speed
 * differs.  Needs a shape with a tensor-core attention (else
 * AVSG_ERR_UNSUPPORTED at create); ignored with AVSG_FLAG_NO_REUSE. */
#define AVSG_FLAG_REQUEST_GATHER 2u

typedef struct avsg_handle_s* avsg_handle;

/*
 * Shape of one handle.  Units are ordered request-major: unit = r * H + h.
 * Host K is laid out [R][H][num_entries][entry_tokens][head_dim] bf16, host V
 * [R][H][num_entries][entry_tokens][v_dim] bf16: one entry of a unit is a
 * contiguous row of entry_tokens tokens (a head-wise page when > 1, Spin page
 * section 2B "head-wise physical pages").  The first initial_entries entries
 * of every unit are live at create (all num_entries when 0); selected ids must
 * be below the live count, which avsg_append raises by one per call.
 */
typedef struct avsg_config {
  int32_t num_requests;        /* R >= 1 */
  int32_t num_kv_heads;        /* H >= 1 */
  int32_t q_per_kv;            /* G: query heads per kv-head (1, 2, 4, 8 or 16) */
  int32_t entry_tokens;        /* tokens per entry: 1 (token) .. 64 (page) */
  int32_t head_dim;            /* D: K row width, multiple of 8 */
  int32_t v_dim;               /* Dv: V row width (== head_dim when kv_shared) */
  int32_t kv_shared;           /* 1: V is the K row itself (latent cache) */
  int32_t reserved0;           /* must be 0 */
  int64_t num_entries;         /* entries per unit the host arrays hold, 1 .. 2^31 - 1 */
  int32_t buffer_slots;        /* B: device slots per unit */
  int32_t max_select;          /* largest k accepted by avsg_step */
  int32_t max_tokens_per_step; /* largest n_tok (1 .. 8) */
  float softmax_scale;         /* 0 selects 1/sqrt(head_dim) */
  uint32_t flags;              /* AVSG_FLAG_* */
  int32_t initial_entries;     /* entries live at create, 0 .. num_entries (0: all of
                                  them); avsg_append adds one per unit per call */
} avsg_config;

typedef struct avsg_stats {
  uint64_t steps;           /* steps enqueued (host count) */
  uint64_t selected;        /* selected ids, summed over units and tokens */
  uint64_t unique_selected; /* distinct ids per unit and step (the union), summed */
  uint64_t hits;            /* distinct selected ids that were resident */
  uint64_t misses;          /* distinct selected ids copied from host */
  uint64_t miss_bytes;      /* host bytes copied into the buffer */
  int32_t device_error;     /* 0, or the AVSG_ERR_* code latched on the device */
  int32_t error_unit;       /* unit of that error, or -1 */
  int32_t error_position;   /* flat position (token * k + j) of that error, or -1 */
  int32_t reserved;
} avsg_stats;

typedef struct avsg_info {
  uint64_t device_bytes;    /* device memory held by the handle */
  int32_t hash_capacity;    /* per-unit open-addressing table entries */
  int32_t miss_set_capacity;/* per-unit per-step miss-set entries */
  int32_t attn_splits;      /* split-K partitions per (unit, token) at max_select */
  int32_t gather_ctas;      /* CTAs of the miss gather */
  int32_t num_sms;          /* SMs of the device */
  int32_t host_registered;  /* 1 if create registered the host KV itself */
} avsg_info;

/*
 * Per-kernel device time (ms), accumulated over the steps enqueued while
 * profiling was on: CUDA events recorded just before and after each kernel on
 * the stream it runs on (the events themselves keep consecutive kernels from
 * overlapping their launches).  launches[i] counts the timed launches.
 */
#define AVSG_KERNEL_MATCH 0
#define AVSG_KERNEL_RESERVE 1
#define AVSG_KERNEL_GATHER 2
#define AVSG_KERNEL_ATTENTION 3      /* single pass, or the pass over hit rows */
#define AVSG_KERNEL_ATTENTION_MISS 4 /* pass over miss rows */
#define AVSG_KERNEL_COMMIT 5         /* hash-table update */
#define AVSG_KERNEL_FINISH 6         /* reserved (the miss pass merges the two passes) */
#define AVSG_KERNEL_PLACE 7          /* staged missed rows into their slots */
#define AVSG_NUM_KERNELS 8
typedef struct avsg_kernel_times {
  double ms[AVSG_NUM_KERNELS];
  uint64_t launches[AVSG_NUM_KERNELS];
} avsg_kernel_times;

/*
 * avsg_create -- build a handle.
 *   cfg     : shape (copied).
 *   host_k  : host K rows, layout above; owned by the caller, must outlive the
 *             handle and must not change while steps run.
 *   host_v  : host V rows, or NULL when cfg->kv_shared.
 *   out     : receives the handle.
 * Host memory already allocated mapped (cudaHostAlloc(Mapped) or
 * avsg_host_alloc) is used in place; any other memory is registered with
 * cudaHostRegister(Mapped | ReadOnly) and unregistered by avsg_destroy.
 * Device memory is allocated on the current device; the buffer starts empty.
 * Errors: INVALID_ARG, CAPACITY (max_tokens_per_step * max_select > buffer_slots),
 * UNSUPPORTED, CUDA.  On error *out is NULL and nothing is held.
 */
int avsg_create(const avsg_config* cfg, const void* host_k, const void* host_v,
                avsg_handle* out);

/* avsg_destroy -- synchronise, free device memory, unregister host memory if
 * create registered it.  NULL is accepted. */
int avsg_destroy(avsg_handle h);

/*
 * avsg_step -- one decode step (one MTP iteration when n_tok > 1).
 *   t          : step index, >= 0 and strictly larger than the previous call's.
 *   n_tok, k   : query tokens (1 .. max_tokens_per_step) and selected entries
 *                per token (0 .. max_select); n_tok * k <= buffer_slots.
 *   d_sel      : device int32 [R][H][n_tok][k], ids in [0, num_entries),
 *                distinct within one token's list (may repeat across tokens).
 *   d_q        : device fp32 [R][H][n_tok][G][D].
 *   d_out      : device fp32 [R][H][n_tok][G][Dv]; attention of each query
 *                head over the rows of its token's selected entries
 *                (softmax(scale * q.K) V, fp32 accumulation); zeros when k = 0.
 *   d_slot_map : device int32 [R][H][n_tok][k] or NULL: buffer slot of each
 *                selected id, input order.
 *   d_hit      : device uint8 [R][H][n_tok][k] or NULL: 1 if the id was
 *                resident before the step.
 *   stream     : cudaStream_t (NULL = legacy default stream).
 * Host-side errors (INVALID_ARG, CAPACITY, BAD_STEP, LATCHED) change nothing.
 * Device-detected errors (BAD_SELECTION) are latched before any buffer state
 * changes: the rest of the step, and every later step, does nothing on the
 * device until avsg_clear_error; avsg_get_stats reports them.
 * With AVSG_FLAG_NO_REUSE the buffer is bypassed: every selected row is copied
 * to a staging area and d_slot_map receives the staging index (tok * k + j),
 * d_hit zeros; ids are range-checked but repeats are not rejected.
 */
int avsg_step(avsg_handle h, int32_t t, int32_t n_tok, int32_t k, const int32_t* d_sel,
              const float* d_q, float* d_out, int32_t* d_slot_map, uint8_t* d_hit,
              void* stream);

/*
 * avsg_step_host -- avsg_step with HOST buffers (same shapes).  Copies the
 * selection and queries to device staging owned by the handle, runs the step,
 * and copies d_out (and the slot map / hit flags when non-NULL) back, all
 * enqueued on `stream`; the results are valid after the stream synchronises.
 * Pinned host buffers make the copies asynchronous.
 */
int avsg_step_host(avsg_handle h, int32_t t, int32_t n_tok, int32_t k, const int32_t* h_sel,
                   const float* h_q, float* h_out, int32_t* h_slot_map, uint8_t* h_hit,
                   void* stream);

/*
 * Offload of a decode step's new KV (Spin page, section 2A, the Offload
 * operation): writes one new entry per unit into the host arrays at entry
 * index `live` (the current live count) and makes it selectable from the next
 * step on.  d_k: device bf16 [R][H][entry_tokens * head_dim]; d_v: device bf16
 * [R][H][entry_tokens * v_dim], NULL when kv_shared.  One strided copy per
 * array, device to host, enqueued on `stream` (ordered before later steps on
 * that stream); the buffer is not touched (a new entry is a miss until it is
 * selected).  For paged entries, a page is appended once it is full.
 * Works the same with AVSG_FLAG_NO_REUSE (both paths read host rows by id).
 * Returns CAPACITY when all num_entries entries are live, INVALID_ARG for
 * NULL rows, CUDA if the copy cannot be enqueued.
 */
int avsg_append(avsg_handle h, const void* d_k, const void* d_v, void* stream);

/*
 * Buffer elasticity (Spin page, section 2B): the buffer of each unit is sized
 * per step, split into mandatory slots (the current step's selection) and
 * buffer slots kept for temporal locality, under a system-wide budget.
 * avsg_set_budget gives every unit u a budget of usable slots, slots_per_unit
 * (host int32 [R][H]), each in 1 .. buffer_slots; it applies from the next
 * step on (enqueued on `stream`).  Entries held in slots at or above a lowered
 * budget are dropped (a later selection of them is a miss); the reservation
 * takes only slots below the budget.  A step needs n_tok * k <= every unit's
 * budget (else CAPACITY).  At create every budget is buffer_slots; avsg_reset
 * keeps the budgets.  Not available with AVSG_FLAG_NO_REUSE (UNSUPPORTED).
 */
int avsg_set_budget(avsg_handle h, const int32_t* slots_per_unit, void* stream);

/*
 * A planner for avsg_set_budget (host only, no handle): splits total_slots over
 * num_units units, each first given `mandatory` slots (the largest n_tok * k
 * it will run), the rest in proportion to weights[u] >= 0 (equal shares when
 * weights is NULL or all zero; the remainder of an equal split goes to the
 * lowest units), each capped at max_slots (buffer_slots).  Slots above a cap
 * stay unassigned.  out: host int32 [num_units].  Returns CAPACITY when
 * total_slots < num_units * mandatory, INVALID_ARG for bad arguments.
 */
int avsg_plan_budget(int64_t total_slots, int32_t num_units, int32_t mandatory, int32_t max_slots,
                     const float* weights, int32_t* out);

/* avsg_get_stats -- synchronise the last stream used and read the counters. */
int avsg_get_stats(avsg_handle h, avsg_stats* out);

/* avsg_info -- static facts about the handle. */
int avsg_get_info(avsg_handle h, avsg_info* out);

/*
 * avsg_read_state -- synchronise and copy one unit's buffer state to host:
 *   tag [B] int32 (resident id or -1), last_step [B] int32 (-1 when never
 *   used), k_rows [B][entry_tokens * D] bf16, v_rows [B][entry_tokens * Dv]
 *   bf16 (NULL when kv_shared).  Any output may be NULL.
 */
int avsg_read_state(avsg_handle h, int32_t unit, int32_t* tag, int32_t* last_step,
                    void* k_rows, void* v_rows);

/* avsg_reset -- empty every buffer, forget the last t, zero the counters
 * (enqueued on `stream`). */
int avsg_reset(avsg_handle h, void* stream);

/* avsg_clear_error -- synchronise, drop a latched device error and the
 * per-step scratch it left; the buffer state is as before the failed step. */
int avsg_clear_error(avsg_handle h);

/* avsg_profile -- enable (1) / disable (0) per-kernel event timing; enabling
 * zeroes the accumulated times. avsg_profile_read synchronises and reads. */
int avsg_profile(avsg_handle h, int32_t enable);
int avsg_profile_read(avsg_handle h, avsg_kernel_times* out);

/*
 * avsg_attention_noalloc -- the attention of avsg_step over rows the caller
 * already holds on the device, allocating nothing.  The pages have no
 * counterpart: this exists for callers that cannot call cudaMalloc (code
 * running inside another framework's memory pool or allocator budget, or a
 * serving process that must not allocate once it runs).
 *   d_k_rows   : device bf16 [num_units][rows_per_unit][entry_tokens][head_dim].
 *   d_v_rows   : device bf16 [num_units][rows_per_unit][entry_tokens][v_dim],
 *                ignored (may be NULL) when kv_shared (V is the K row).
 *   d_index    : device int32 [num_units][n_tok][k], row of each selected
 *                entry, each in [0, rows_per_unit).  Repeats within one
 *                (unit, token) list are not detected: such a row counts once
 *                per occurrence (avsg_step rejects them).
 *   d_q, d_out : as in avsg_step.  softmax_scale 0 selects 1/sqrt(head_dim).
 * Shapes: those avsg_create accepts for attention; num_units <= 4096 and
 * k <= rows_per_unit (AVSG_ERR_CAPACITY beyond), n_tok <= 8.
 * Scratch: a fixed 8 MiB device array inside the library, held by every GPU
 * that loads it until the process exits.  The first call on a device looks
 * up that array's address (cudaGetSymbolAddress); make the first call before
 * any stream capture.  Every call shares the array and clears what must start
 * at zero; calls that overlap on the GPU race, so serialise them.
 * An index outside [0, rows_per_unit) makes the call fill d_out with NaN.
 * Returns after enqueueing on `stream`.  The argument errors (INVALID_ARG,
 * CAPACITY, UNSUPPORTED) are found before anything is enqueued and change
 * nothing; after AVSG_ERR_CUDA part of the work may have been enqueued and
 * d_out is undefined.
 */
int avsg_attention_noalloc(int32_t num_units, int32_t rows_per_unit, int32_t q_per_kv,
                           int32_t head_dim, int32_t v_dim, int32_t entry_tokens,
                           int32_t kv_shared, int32_t n_tok, int32_t k, const void* d_k_rows,
                           const void* d_v_rows, const int32_t* d_index, const float* d_q,
                           float* d_out, float softmax_scale, void* stream);

/* Pinned, mapped, portable host memory for the KV cache (cudaHostAlloc). */
int avsg_host_alloc(size_t bytes, void** out);
int avsg_host_free(void* p);

/*
 * avsg_read_rows -- a measurement aid: reads n rows at scattered positions and
 * discards them, to measure the ceiling of the step's row reads.  The
 * attention reads the selected entries' rows from slots scattered over the
 * device buffer, and the miss gather reads the missed entries' rows from ids
 * scattered over the host store (AVSG page, arxivdaily 2609.37538, English
 * abstract: only the selected entries are read; only the misses cross the
 * host link); the rate of this read alone, at the same row size, bounds both.
 *   src      : rows [num_rows][row_bytes], device memory or the device pointer
 *              of mapped host memory; 16-byte aligned.
 *   row_bytes: a multiple of 16.
 *   d_idx    : device int32 [n], the rows to read; an index outside
 *              [0, num_rows) is skipped.
 *   ctas     : grid size, 0 for 4 per SM.
 *   d_sink   : device uint32 the kernel may write (it practically never does).
 * Enqueued on `stream`; INVALID_ARG for bad arguments, CUDA if the launch fails.
 */
int avsg_read_rows(const void* src, int64_t num_rows, int64_t row_bytes, const int32_t* d_idx,
                   int64_t n, int32_t ctas, uint32_t* d_sink, void* stream);

/*
 * Paged device cache.  For K and V that stay on the device -- a draft model's
 * layers, layers that are not offloaded -- and for drafted tokens that are not
 * part of the host store yet: block tables and slot maps built on the GPU from
 * request lengths, rotary positions written straight into the pages, attention
 * for draft trees (or chains, or prompt chunks) over the pages, and the keep
 * of the accepted drafts.  A step is
 *   avsg_page_plan     once: tables, slots and positions of the new tokens
 *   avsg_rotary_write  per layer: q rotated, k rotated and stored, v stored
 *   avsg_tree_attention per layer
 *   avsg_tree_keep     once, for all layers, when the drafts are verified
 * and may be captured into one CUDA graph: no call allocates, synchronises or
 * reads a length on the host.
 *
 * Layout.  d_k and d_v are [num_layers][num_pages][H][page_tokens][D]: one
 * page of one kv-head is contiguous (Spin page, section 2B, head-wise pages).
 * Token j of request r is row j % page_tokens of page
 * d_tables[r][j / page_tokens]; its slot is page * page_tokens + row.  The
 * first d_len[r] tokens of a request are committed; a step's new tokens follow
 * them.  New tokens are ragged: request r owns rows d_first[r] ..
 * d_first[r + 1] of every per-token array.  Free page ids are a stack:
 * d_free[0 .. d_free_count[0]).
 *
 * Errors.  Host checks return a code and enqueue nothing.  What only the
 * device can see (a page id outside the pool, too few free pages, a path that
 * is not increasing) is latched in d_error = {code, request, position}; the
 * first error stays, and every later call on the same d_error does nothing on
 * the device until the caller zeroes it.  avsg_page_plan calls on one d_error
 * must not run at the same time.  All memory is the caller's, on the
 * current device (INVALID_ARG for pages of another one), and must stay valid
 * until the enqueued work is done.  A page belongs to one request unless
 * avsg_page_fork shares it; a cache with shared pages is kept by
 * avsg_tree_keep_shared, as avsg_tree_keep would give a shared page back twice.  Calls on several streams are independent
 * as long as nothing that one of them writes is used by another at a time.
 * That holds for a d_error of several caches too: an error that one latches
 * may stop another's call part of the way, but for avsg_page_fork and
 * avsg_page_compact, which happen as a whole or not at all.
 */
#define AVSG_BF16 0
#define AVSG_F16 1

typedef struct avsg_pages {
  int32_t num_requests; /* R, 1 .. 8192 */
  int32_t num_layers;   /* >= 1 */
  int32_t num_pages;    /* pages of the pool; num_pages * page_tokens < 2^31 */
  int32_t num_kv_heads; /* H */
  int32_t page_tokens;  /* a power of two, 1 .. 256 */
  int32_t head_dim;     /* D, a multiple of 8 */
  int32_t max_pages;    /* columns of d_tables */
  int32_t dtype;        /* AVSG_BF16 or AVSG_F16 */
  void* d_k;            /* 16-byte aligned */
  void* d_v;
  int32_t* d_tables;    /* [R][max_pages] */
  int32_t* d_len;       /* [R] committed tokens */
  int32_t* d_free;      /* [num_pages] stack of free page ids */
  int32_t* d_free_count;/* [1] */
  int32_t* d_error;     /* [4], zeroed by the caller at first; the fourth is the library's */
} avsg_pages;

/*
 * avsg_page_plan -- tables, slots and positions of a step's new tokens.
 *   d_new   : int32 [R], new tokens per request (0 is allowed).
 *   d_mask  : uint64 [num_mask] or NULL: ancestors of each draft (see
 *             avsg_tree_attention); position = len + depth, with depth the
 *             number of bits - 1.  NULL, a zero word, or a request with more
 *             than 64 new tokens, whose words are not looked at: len + index.
 *   capacity: entries of d_slot and d_pos.
 *   d_first : int32 [R + 1], receives the exclusive sum of d_new.
 *   d_slot  : int32 [capacity], receives each token's slot, -1 behind the last.
 *   d_pos   : int32 [capacity], receives positions, 0 behind the last.
 *   d_free_count_out: int32 [1], may be d_free_count itself.
 * Pages are taken from the top of the stack in request order and entered in
 * d_tables; entries that do not change are not written.  Latched errors
 * (CAPACITY: too few free pages, table columns, entries or masks; BAD_SELECTION: a
 * negative length or a page id outside the pool) leave everything as it was.
 */
int avsg_page_plan(const avsg_pages* p, const int32_t* d_new, const uint64_t* d_mask,
                   int32_t num_mask, int32_t capacity, int32_t* d_first, int32_t* d_slot, int32_t* d_pos,
                   int32_t* d_free_count_out, void* stream);

/*
 * avsg_rotary_frequencies -- host only: the table of avsg_rotary_write.
 *   out[i], i < rot_dim / 2: turns per position of pair i as a 64-bit binary
 *   fraction (2^64 = one turn) of w_i = base^(-2i / rot_dim), scaled for long
 *   contexts: by 1 / factor when original is 0; else pairs that turn at least
 *   high_turns times in `original` tokens keep w_i, pairs below low_turns get
 *   w_i / factor, with a ramp between that is linear in the turns (a model
 *   whose ramp is linear in the pair's index needs a table of its own).
 */
int avsg_rotary_frequencies(int32_t rot_dim, double base, double factor, double low_turns,
                            double high_turns, double original, uint64_t* out);

typedef struct avsg_rotary {
  int32_t num_tokens;         /* T */
  int32_t num_q_heads;        /* a multiple of num_kv_heads */
  int32_t rot_dim;            /* rotated values per head, even, 0 .. D */
  int32_t rot_offset;         /* first rotated value; the others keep theirs */
  int32_t interleaved;        /* 1: pairs (2i, 2i + 1); 0: (i, i + rot_dim / 2) */
  int32_t q_f32;              /* 1: d_q_out is fp32 (avsg_step's q), else the cache's type */
  int32_t tokens_per_request; /* n: d_q_out is [T / n][H][n][G][D]; 1 is [T][heads][D] */
  int32_t layer;
  int64_t q_stride, k_stride, v_stride; /* values between tokens' rows */
  float magnitude;            /* factor on cos and sin (1 for none), finite */
  int32_t reserved0;          /* must be 0 */
  const void* d_q;            /* [T] rows of num_q_heads * D values, the cache's type */
  const void* d_k;            /* [T] rows of H * D */
  const void* d_v;            /* [T] rows of H * D */
  const uint64_t* d_freq;     /* [rot_dim / 2] */
  const int32_t* d_pos;       /* [T] */
  const int32_t* d_slot;      /* [T] or NULL: slot t for token t */
  void* d_q_out;
} avsg_rotary;

/*
 * avsg_rotary_write -- rotates q and k by their tokens' positions, writes q to
 * d_q_out and k, v to their slots of the given layer.  Angles are exact at any
 * int32 position; arithmetic is fp32, rounded once.  A token with slot -1 is
 * skipped whole (padding); a slot past the pool is latched (BAD_SELECTION), its
 * token not written, the call's others written or not.  Slots must be distinct.  d_q_out may be d_q when the types
 * agree, tokens_per_request is 1 and q_stride is num_q_heads * D; otherwise
 * outputs must not overlap inputs.  With page_tokens 1, num_pages T and no
 * slots, d_k and d_v are the [R][H][D] rows avsg_append takes, and with q_f32
 * and tokens_per_request n_tok, d_q_out is the d_q of avsg_step.
 */
int avsg_rotary_write(const avsg_pages* p, const avsg_rotary* r, void* stream);

/*
 * avsg_tree_attention -- attention of a step's new tokens over the pages.
 * Per new token and query head:  s = scale q.k;  softcap > 0: s = softcap *
 * tanh(s / softcap);  d_slopes: s -= slope * (position of q - position of k);
 * out = softmax(s) v over the visible keys, lse = log of the sum of exp(s).
 * New token i of a request sees every committed token and, of its new ones,
 * those in its mask word (bit j: new token j of the same request; an ancestor
 * mask holds the token's own bit).  d_mask NULL, or a request with more than
 * 64 new tokens, whose words are not looked at: the new tokens up to itself (a
 * chain, or a prompt chunk).
 * Positions: a committed token's index; a new token's len + number of mask
 * bits - 1 (bits past the request's tokens stand for no key, but count), len + i
 * for a chain or a zero word.  window > 0: only keys with
 * position of q - position of k < window.  The new tokens' own K and V must
 * be in the pages (avsg_rotary_write).  A row without a visible key gives
 * zeros and -infinity.  What a row does not see does not reach it, whatever
 * it holds; neither does what lies in the pages behind the last new token.
 * A value of V that is not finite makes the results that see it not finite: an
 * infinity, or NaN where its weight rounds to 0 in the cache's type.
 * Scores, sums and outputs are fp32; q is read and the weights are multiplied
 * with V in the cache's type (half a step each), and so is the result.
 * Outputs must not overlap inputs.
 */
typedef struct avsg_tree {
  int32_t num_tokens;   /* rows of d_q, d_out and d_lse (at least d_first[R]; the
                           rows behind d_first[R] are left as they are) */
  int32_t q_per_kv;     /* G: query heads per kv-head, 1 .. 64 */
  int32_t max_new;      /* no request has more new tokens (else CAPACITY is latched) */
  int32_t layer;
  int32_t window;       /* 0: none */
  float softmax_scale;  /* 0 selects 1/sqrt(D); below 2^126 */
  float softcap;        /* 0: none; below 2^127; softmax_scale / softcap below 2^126 */
  int32_t reserved0;    /* must be 0 */
  int64_t q_stride;     /* values between tokens of d_q, even */
  const void* d_q;      /* rows of [H][G][D], the cache's type, 4-byte aligned */
  const int32_t* d_first; /* [R + 1] */
  const uint64_t* d_mask; /* [tokens] or NULL */
  const float* d_slopes;  /* [H * G] or NULL */
  void* d_out;          /* [num_tokens][H][G][D], the cache's type, 16-byte aligned */
  float* d_lse;         /* [num_tokens][H][G] or NULL */
  void* d_work;         /* 256-byte aligned, any contents */
  size_t work_bytes;    /* at least avsg_tree_attention_workspace */
} avsg_tree;

/*
 * Bytes of d_work for the device of p->d_k.  The size depends on D, q_per_kv
 * and max_new, not on lengths or the pool.  Calls that may run at the same time (two
 * streams, two graphs) need a workspace each.
 */
int avsg_tree_attention_workspace(const avsg_pages* p, int32_t q_per_kv, int32_t max_new,
                                  size_t* bytes);

/*
 * D of 64, 128 or 256 (UNSUPPORTED else).  Latched errors: BAD_SELECTION (a
 * page id outside the pool, a negative length, rows past num_tokens; position
 * = the key), CAPACITY (more than max_new new tokens, or than the table
 * holds), TIMEOUT (a wait inside the kernel gave up after about two seconds);
 * d_out and d_lse of such a call are undefined, nothing else is written.
 */
int avsg_tree_attention(const avsg_pages* p, const avsg_tree* t, void* stream);

/*
 * avsg_tree_keep -- keeps the accepted drafts and ends requests.
 *   d_first : as written by the step's avsg_page_plan.
 *   d_keep  : int32 [R]: number of kept new tokens, or -1: the request ends
 *             (its length becomes 0 and all its pages are free).
 *   d_path  : int32 [num_path] or NULL: the kept tokens' indices within their
 *             request, strictly increasing, at d_path[d_first[r] + i]; NULL
 *             keeps the first d_keep[r].
 * Row len + path[i] moves to len + i in every layer; d_len_out (may be d_len)
 * receives the new lengths; the pages past them return to the stack in the
 * reverse order of taking, and d_free_count_out (may be d_free_count) counts
 * them.  Latched errors (BAD_SELECTION: a bad count, path or page id;
 * CAPACITY: more pages than the pool, or more tokens than num_path) leave
 * everything as it was.
 */
int avsg_tree_keep(const avsg_pages* p, const int32_t* d_first, const int32_t* d_path,
                   int32_t num_path, const int32_t* d_keep, int32_t* d_len_out, int32_t* d_free_count_out,
                   void* stream);

/*
 * Rotary positions of several axes (time, height, width of an image's or a
 * video's patches): as avsg_rotary_write, but r->d_pos is int32 [num_axes][T]
 * and pair i of a head turns by the position on axis d_axis[i] (device int32
 * [rot_dim / 2], each in [0, num_axes): else BAD_SELECTION is latched and nothing
 * is written).
 */
int avsg_rotary_write_axes(const avsg_pages* p, const avsg_rotary* r, int32_t num_axes,
                           const int32_t* d_axis, void* stream);

/*
 * Shared pages.  Requests with a common beginning (samples of one prompt, beams,
 * a batch behind one system prompt) hold the same full pages: d_shares[page],
 * int32 [num_pages], counts the requests that hold a page beyond the first; it is 0 for
 * free pages and for pages of one request, so a new cache's is all zeros.
 * avsg_page_plan, avsg_rotary_write and both attentions take such a cache as
 * it is: new tokens never lie in a shared page.
 *
 * avsg_page_fork -- requests continue as copies of others.
 *   d_parent : int32 [R]: request r becomes what request d_parent[r] was
 *              (itself: it stays; -1: it ends, with length 0 and no pages).
 *              Several may have the same parent, and a parent may itself
 *              become another: samples, beams that replace beams, ends.
 * The full pages of the parent's committed tokens are shared.  Its partly
 * filled last page stays with the parent if that stays, else goes to its
 * lowest child; every other child takes a page from the stack (in request
 * order) and the filled rows are copied there in all layers.  Pages that
 * nobody holds any more go back after that, in the reverse order of taking, listed by
 * the highest request that held them and by column.  Tables, lengths, shares, stack and count
 * change in place; table entries behind a request's pages are left as they are.  New tokens that are
 * not committed (avsg_tree_keep) are not looked at: fork between steps.
 * Latched errors (BAD_SELECTION: a parent, length, page id or count out of
 * range; CAPACITY: too few free pages or table columns, or more pages than the pool) leave everything as
 * it was.  d_work: 256-byte aligned, any contents; max_pages up to 2^30.
 */
int avsg_page_fork_workspace(const avsg_pages* p, size_t* bytes);
int avsg_page_fork(const avsg_pages* p, const int32_t* d_parent, int32_t* d_shares, void* d_work,
                   size_t work_bytes, void* stream);

/*
 * avsg_tree_keep_shared -- avsg_tree_keep for a cache with shared pages.  A
 * request that ends here (d_keep -1) and holds a shared page latches
 * BAD_SELECTION, and everything stays as it was: such requests end by avsg_page_fork.
 */
int avsg_tree_keep_shared(const avsg_pages* p, const int32_t* d_shares, const int32_t* d_first,
                          const int32_t* d_path, int32_t num_path, const int32_t* d_keep, int32_t* d_len_out,
                          int32_t* d_free_count_out, void* stream);

/*
 * avsg_page_compact -- the pages in use move to the front of the pool.
 * Pages in use are those that are not on the stack, whoever holds them.  With
 * n of them, the i-th of those at or above n (by id) moves to the i-th free
 * id below n, whole and in all layers; pages above n can then be given to something
 * else, or the pool cut off there.  Compact between steps, as for the fork:
 * a page that avsg_page_plan took for tokens that are not committed yet is in
 * use and moves, but its entry behind the committed tokens and the step's
 * slots keep the old id, under which another page may lie from then on (a
 * caller who holds pages of its own finds them by d_map).
 *   d_shares, d_shares_out : as above, both or neither NULL.
 *   d_tables_out : [R][max_pages], receives the tables (entries behind a
 *                  request's pages as they were).
 *   d_free_out   : [num_pages], receives the stack: pages are taken from n upward
 *                  (entries at or above the count, which stays, as they were).
 *   d_map        : int32 [num_pages], receives each page's new id, -1 for a free one.
 * Each output may be the input itself (d_tables, d_free, d_shares); outputs that are not
 * leave the input as it was.  Latched errors (BAD_SELECTION: an id out of
 * range or twice on the stack, a held page that is free, a negative length; CAPACITY: more tokens than the
 * table holds) leave everything as it was.  d_work: 256-byte aligned, any contents; max_pages up to 2^30.
 */
int avsg_page_compact_workspace(const avsg_pages* p, size_t* bytes);
int avsg_page_compact(const avsg_pages* p, const int32_t* d_shares, int32_t* d_shares_out, int32_t* d_tables_out,
                      int32_t* d_free_out, int32_t* d_map, void* d_work, size_t work_bytes, void* stream);

/* Groups of requests with a common prefix, and their new tokens in order. */
typedef struct avsg_prefixes {
  int32_t num_tokens;   /* entries of d_token and d_request: at least the step's new tokens */
  int32_t reserved0;    /* must be 0 */
  int32_t* d_leader;    /* [R] the lowest request of the group, the request itself if it is alone */
  int32_t* d_shared;    /* [R] tokens of the group's prefix, whole pages; 0: alone */
  int32_t* d_first;     /* [R + 1] first place of the group that the request leads (exclusive sum) */
  int32_t* d_token;     /* [num_tokens] the token in each place, -1 behind the last */
  int32_t* d_request;   /* [num_tokens] its request, -1 behind the last */
} avsg_prefixes;

/*
 * avsg_prefix_find -- finds the step's groups from the tables (once per step,
 * after avsg_page_plan; every layer's attention uses them).  Requests with new
 * tokens whose tables begin with the same page form a group, if the full
 * pages that all of them have in common hold at least min_tokens committed
 * tokens (and there are two members).  d_first: as written by avsg_page_plan.
 * Latched errors (BAD_SELECTION: a negative length, bad first tokens, a first
 * page outside the pool; CAPACITY: more full pages than columns) leave the outputs as they were.
 * d_work: 256-byte aligned, any contents; max_pages up to 2^30.
 */
int avsg_prefix_find_workspace(const avsg_pages* p, size_t* bytes);
int avsg_prefix_find(const avsg_pages* p, const int32_t* d_first, int32_t min_tokens, const avsg_prefixes* x,
                     void* d_work, size_t work_bytes, void* stream);

/*
 * avsg_prefix_attention -- avsg_tree_attention in which the keys of a group's
 * prefix are read and multiplied once for the new tokens of all its members.
 * The same results up to rounding: masks, chains, positions, caps, biases and
 * windows are those of avsg_tree_attention, whatever the groups are.
 *   t : as for avsg_tree_attention; t->d_work and t->work_bytes go by this
 *       operator's workspace, which grows with the tokens.
 *   x : the groups, as avsg_prefix_find wrote them for these tables, lengths
 *       and first tokens.  Latched (BAD_SELECTION): indices out of range, and
 *       a token of a request with a prefix (d_shared[r] > 0) that is not in the
 *       list of a group whose leader has a prefix of that length.  Other
 *       arrays that do not fit (a member whose first pages are not the
 *       leader's) give undefined results.
 * Errors and rounding as avsg_tree_attention; what a call that latches an error wrote is undefined.
 */
int avsg_prefix_attention_workspace(const avsg_pages* p, int32_t q_per_kv, int32_t max_new, int32_t num_tokens,
                                    size_t* bytes);
int avsg_prefix_attention(const avsg_pages* p, const avsg_tree* t, const avsg_prefixes* x, void* stream);

/* Error text, and the cudaError_t behind the last AVSG_ERR_CUDA of a handle. */
const char* avsg_strerror(int code);
int avsg_cuda_error(avsg_handle h);

#ifdef __cplusplus
}
#endif

#endif /* AVSG_H_ */
