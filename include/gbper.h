/*
 * gbper.h -- GPU-resident prioritized experience replay (PER) on one GB300 (sm_103a).
 *
 * A C ABI over plain pointers and sizes.  Every transition, priority and batch lives in device
 * memory; the library owns the replay ring and the priority trees, the caller owns every input
 * and output buffer it passes.  No call takes or returns a torch type.
 *
 * Sources (cited by page title and section):
 *   "GPU-Resident Prioritized Experience Replay" (foxhunt design document): Architecture,
 *     Sampling Kernels (Proportional, Rank-based), Priority update, Experience Insertion,
 *     Error Handling & Fallback.
 *   "Putting prioritized replay's segment tree on a GPU": The Tree Under Every Prioritized
 *     Replay, Sampling Is a Descent, Second Port: Make the Update GPU-Shaped.
 *   "True Single-Graph Implementation Plan": Task 2 (padded row gather, int64 indices),
 *     Task 3 (gather straight into the trainer's buffers), Task 4 (device-side counters),
 *     Task 5 (PER calls as stream work that a CUDA graph can capture).
 *
 * Conventions shared by every call
 *   - Streams.  `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *     stream).  Work is enqueued on it; no call below synchronises the host unless its
 *     comment says so (per_total, per_min, per_status_device, per_read_state).
 *   - Device pointers.  Arguments named d_* are device addresses (cudaMalloc or the caching
 *     allocator of a framework) on the device that was current at per_create.  They must stay
 *     valid until the enqueued work has run.  Row arrays must be 4-byte aligned; 16-byte
 *     alignment together with a row length that is a multiple of 4 floats enables the
 *     vectorised copy paths.
 *   - Errors.  Every call returns a per_status.  Invalid host-side arguments return
 *     PER_ERR_INVALID_ARG before anything is enqueued.  A failed CUDA call returns
 *     PER_ERR_CUDA; per_last_error() then describes it.  Conditions only the device can see
 *     (an update index outside the filled slots, a bounded wait that ran out) never trap or
 *     abort: the kernel skips the offending element and sets a bit in the device error word,
 *     which per_status_device() reads and clears.  Nothing falls back to the CPU.
 *   - Concurrency.  One handle is driven from one host thread at a time, and its calls are
 *     ordered by the caller (one stream, or explicit events across streams).
 */
#ifndef GBPER_H
#define GBPER_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct per_buffer per_buffer; /* opaque; owned by the library */

typedef enum {
    PER_OK = 0,
    PER_ERR_INVALID_ARG = 1, /* rejected on the host; nothing was enqueued */
    PER_ERR_OOM = 2,         /* device allocation in per_create failed */
    PER_ERR_CUDA = 3,        /* a CUDA runtime call failed; see per_last_error */
    PER_ERR_EMPTY = 4,       /* per_sample / per_min on a buffer with no filled slot */
    PER_ERR_DEVICE_FLAG = 5, /* per_status_device: the device error word was non-zero */
    PER_ERR_TIMEOUT = 6      /* a bounded device-side wait gave up (reported as a flag bit) */
} per_status;

/* Sampling modes ("GPU-Resident Prioritized Experience Replay", Sampling Kernels). */
enum {
    PER_MODE_PROPORTIONAL = 0, /* P(i) = p_i^alpha / sum_k p_k^alpha, sum tree + min tree */
    PER_MODE_RANK = 1,         /* P(i) proportional to 1 / rank(i)^alpha, rank by raw priority */
    PER_MODE_UNIFORM = 2,      /* P(i) = 1 / size: the plain replay PER replaces; priorities unused */
    PER_MODE_FLAT = 3          /* proportional, located by the pages' own flat design: an inclusive
                                  sum of the leaves rebuilt at each sample and a search per draw
                                  ("Sampling Kernels", Proportional steps 2-3); no tree */
};

/* Bits of the device error word (per_status_device). */
enum {
    PER_DEVFLAG_BAD_INDEX = 1u, /* an update named an index outside [0, size); it was skipped */
    PER_DEVFLAG_TIMEOUT = 2u,   /* a bounded wait gave up; the call's results are not valid */
    PER_DEVFLAG_RANK_STALE = 4u /* rank mode: more slots were written between two samples than the
                                   order merge can take (only reachable by replaying a captured
                                   sample after more writes than at capture); the order is stale */
};

/* per_config.flags */
enum {
    PER_FLAG_RANK_RESORT = 1u, /* rank mode: sort every filled slot at each sample instead of
                                  merging the slots written since the previous one (same order) */
    PER_FLAG_DONES_F32 = 2u    /* per_sample writes dones as float 0.0f / 1.0f (d_dones is float*,
                                  4-byte aligned), the trainer's format ("True Single-Graph
                                  Implementation Plan", Task 3) */
};

typedef struct {
    double alpha;            /* priority exponent, >= 0 */
    double eps;              /* added to |td| before the exponent; > 0 */
    uint32_t mode;           /* PER_MODE_* */
    uint32_t row_stride_out; /* floats per gathered state row, >= state_dim (0: state_dim);
                                columns past state_dim are written as 0.0f */
    uint64_t seed;           /* key of the Philox4x32-10 stream that draws the batches */
    uint32_t flags;          /* PER_FLAG_* bits; others must be 0 */
    uint32_t rebuild_batch;  /* update batches of at least this many entries scatter their
                                priorities and rebuild every tree level instead of climbing from
                                each changed leaf (same result); 0: the crossover measured on
                                GB300 (max(leaves / 128, 1024) proportional; rank mode
                                always scatters), and smaller batches too while recent
                                updates crowded a subtree (see per_update_priorities);
                                UINT32_MAX: never; any other value: from that size, with
                                no regard to crowding */
    uint32_t element_batch;  /* proportional mode: update batches of fewer entries than this
                                propagate entry by entry, each from its leaf to the root (same
                                result); 0: the crossover measured on GB300 (3: batches of
                                one or two entries); 1: never; UINT32_MAX: always */
    uint32_t reserved;       /* 0 */
} per_config;

/*
 * per_create -- allocate a replay buffer of `capacity` slots holding rows of `state_dim`
 * floats ("GPU-Resident Prioritized Experience Replay", Architecture: a fixed-capacity ring
 * of states, next_states, actions, rewards, dones and priorities; no allocation during
 * training).  Proportional mode also allocates the sum tree (binary64 internal nodes over
 * binary32 leaves p^alpha) and its twin min tree ("Putting prioritized replay's segment tree
 * on a GPU", The Tree Under Every Prioritized Replay); the tree has the next power of two
 * >= capacity leaves, and the extra leaves are never filled.  Rank mode allocates the raw
 * priorities, the sort workspace and the rank CDF, which it computes here.
 * Every later call reuses these allocations.  The device current at this call owns them.
 *   capacity  1 .. 2^31 slots.
 *   state_dim floats per state row, 0 .. 65536.
 *   cfg       copied; NULL means alpha 0.6, eps 1e-6, proportional, stride = state_dim.
 *   out       receives the handle (unchanged on error).
 * Errors: PER_ERR_INVALID_ARG (bad sizes or config), PER_ERR_OOM, PER_ERR_CUDA.
 */
per_status per_create(uint64_t capacity, uint32_t state_dim, const per_config *cfg,
                      per_buffer **out);

/* per_destroy -- synchronise the device, release every allocation and the handle.
 * NULL is accepted and ignored. */
per_status per_destroy(per_buffer *h);

/*
 * per_add -- insert `count` transitions at the ring cursor ("GPU-Resident Prioritized
 * Experience Replay", Experience Insertion): row k goes to slot (cursor + k) mod capacity, so
 * when count > capacity only the last `capacity` rows stay; the cursor wraps and the filled
 * size grows to at most capacity.  Each new slot's raw priority is d_raw_prio[k] or, when
 * d_raw_prio is NULL, the running maximum raw priority ("new experiences get max_priority").
 * Raw priorities pass the clamp of Error Handling & Fallback: NaN becomes eps, +Inf becomes
 * the running maximum as it stood when the call began, values below eps become eps.  The
 * running maximum then takes every new raw priority.  Proportional mode writes the leaves
 * p^alpha (binary64 pow rounded to binary32) and rebuilds the dirty ancestors of both trees
 * level by level ("Putting prioritized replay's segment tree on a GPU", Second Port).
 *   d_states, d_next  [count x state_dim] float, row-major (may be NULL when state_dim = 0).
 *   d_actions [count] uint32, d_rewards [count] float, d_dones [count] uint8.
 *   d_raw_prio [count] float or NULL.
 * count = 0 is a no-op.  No host synchronisation.
 */
per_status per_add(per_buffer *h, uint64_t count, const float *d_states, const float *d_next,
                   const uint32_t *d_actions, const float *d_rewards, const uint8_t *d_dones,
                   const float *d_raw_prio, void *stream);

/*
 * per_sample -- draw a stratified batch of B transitions and gather it into caller buffers.
 * Proportional mode ("GPU-Resident Prioritized Experience Replay", Sampling Kernels,
 * Proportional; "Putting prioritized replay's segment tree on a GPU", Sampling Is a Descent):
 * draw j takes u_j from Philox4x32-10 (counter = (j, call lo, call hi, 0), key = seed, 53-bit
 * uniform from the first two words), mass_j = (j + u_j) * (T / B) with T the root sum, and
 * walks from the root: left when the left child's sum exceeds the mass, otherwise subtract
 * and go right.  A walk that ends past the filled slots is clamped to the last filled slot.
 * The IS weight is w = (n P(i))^-beta / max_w with max_w from the min tree, which equals
 * (p_i^alpha / p_min^alpha)^-beta.
 * Rank mode ("Sampling Kernels", Rank-based): sorts the filled slots by raw priority
 * descending (ties by slot ascending), draws mass_j = (j + u_j) * (c_size / B) with counter
 * tag 1, takes the rank r whose CDF interval c_{r-1} <= mass < c_r holds it, with
 * c_r = sum_{k<=r} k^-alpha, and weights w = (r / size)^(alpha * beta).  The order is kept
 * between calls: when it exists and at most 4096 slots (and at most an eighth of the filled
 * ones, by the host's count of inserted and updated entries) were written since, only those
 * slots are merged back into it; otherwise every filled slot is sorted again.  Both give the
 * same order.
 * Uniform mode (the plain replay that PER replaces, "GPU-Resident Prioritized Experience
 * Replay", Experience Insertion): every filled slot weighs 1, so draw j (counter tag 2) takes
 * mass_j = (j + u_j) * (size / B) and slot floor(mass_j), clamped to the last filled slot;
 * w = 1.
 * Flat mode ("Sampling Kernels", Proportional steps 2-5, the pages' own design): the same draws
 * as proportional mode (tag 0); the call first sums the filled leaves into the inclusive array
 * C[i] = L[0] + ... + L[i] (fixed-point sums with the unit 2^-52 of the largest leaf's binade,
 * each prefix rounded once to binary64), then draw j takes the first slot with
 * C[slot] > mass_j, T = C[size-1], and the same weight with p_min the smallest filled leaf.
 * The sums round differently from the tree's, so slot choices can differ from proportional
 * mode only for masses within rounding distance of a boundary.  Flat mode needs alpha <= 1.
 * Gather ("True Single-Graph Implementation Plan", Task 2/3): row j of d_states and d_next
 * receives the chosen slot's row, padded with 0.0f to row_stride_out floats.
 *   d_idx [B] int64 (required); d_w [B] float; d_states, d_next [B x row_stride_out] float;
 *   d_actions [B] uint32; d_rewards [B] float; d_dones [B] uint8 (float with
 *   PER_FLAG_DONES_F32) -- each may be NULL to skip.
 *   B in 1 .. 2^24.  beta >= 0.
 * The call counter lives on the device, so each call, captured in a graph or not, draws a
 * fresh batch.  PER_ERR_EMPTY when the buffer holds no transition (host-side count).  In rank
 * mode the slot order's length is fixed at launch, so a call made during stream capture while
 * the buffer is not yet full is refused (PER_ERR_INVALID_ARG): capture rank-mode rounds once the
 * ring is full.
 */
per_status per_sample(per_buffer *h, uint32_t B, float beta, int64_t *d_idx, float *d_w,
                      float *d_states, float *d_next, uint32_t *d_actions, float *d_rewards,
                      uint8_t *d_dones, void *stream);

/*
 * per_update_priorities -- write new priorities for a batch from its TD errors
 * ("GPU-Resident Prioritized Experience Replay", Priority update and Error Handling &
 * Fallback): raw = fl32(|td| + eps), NaN -> eps, +-Inf -> the running maximum as it stood
 * when the call began; the leaf becomes raw^alpha.  When an index repeats, the highest batch
 * position wins.  Proportional mode then rebuilds the dirty ancestors of the sum and min
 * trees level by level ("Putting prioritized replay's segment tree on a GPU", Second Port),
 * restricted to the nodes above a changed leaf.  Batches of at least per_config.rebuild_batch
 * entries instead mark each slot's last batch position in a winner word, write the winners and
 * rebuild every level of both trees (the post's level-synchronous rebuild, Measuring the
 * Trade Honestly: O(k + n) beats O(k log n) once k is a large share of n); the trees come out
 * the same.  Smaller batches climb, each warp serving one subtree's entries 32 distinct leaves at
 * a time, one group after the other, so crowding matters: the update kernels report the most
 * entries one subtree received (with the split they used) through mapped host memory, without a
 * synchronisation and a few calls late, and on each new report the next climbs split the tree
 * twice as finely when a subtree held more than 32 entries (up to 2^10 subtrees) and once as
 * coarsely again at 8 or fewer; when even the finest split leaves at least
 * 32 max(2, 5/6 leaves / 2^20) entries in a subtree, the next calls rebuild every level (measured on GB300 at 2^21 leaves,
 * B = 512: up to 465 entries in one subtree climbed in 68-104 us, rebuilt in 33 us), until the
 * counts the rebuild keeps fall below it.  PER_STATE_COUNTERS[4] reads the latest report.  A
 * rebuild_batch other than 0 keeps the size rule alone.  Flat mode writes the leaves only (scatter path
 * always; the next sample sums them).  Rank mode stores raw.  Uniform mode has no
 * priorities: the call checks its arguments and changes nothing.  The running maximum
 * takes every raw priority of the batch.  Indices outside [0, size) are skipped and set
 * PER_DEVFLAG_BAD_INDEX.
 *   d_idx [B] int64, d_td [B] float.  B in 0 .. 2^24 (0 is a no-op).
 */
per_status per_update_priorities(per_buffer *h, uint32_t B, const int64_t *d_idx,
                                 const float *d_td, void *stream);

/*
 * per_rank_refresh -- rank mode: bring the slot order up to date now, the step per_sample takes
 * first ("GPU-Resident Prioritized Experience Replay", Sampling Kernels, Rank-based step 1: the
 * filled slots sorted by raw priority descending, ties by slot ascending).  When the order exists
 * and at most 4096 slots (and at most an eighth of the filled ones) were written since it was
 * made, the written slots are merged into it; otherwise every filled slot is sorted again.  A
 * per_sample that follows with no write in between samples from this order without redoing it;
 * PER_STATE_RANK_ORDER reads it.  A buffer with no filled slot is left as it is.  No host
 * synchronisation.  As for per_sample, a call made during stream capture while the buffer is not
 * yet full is refused.
 * Errors: PER_ERR_INVALID_ARG (not rank mode, or the capture case), PER_ERR_CUDA.
 */
per_status per_rank_refresh(per_buffer *h, void *stream);

/* per_total -- the root of the sum tree (proportional), c_size (rank), size (uniform) or C[size-1]
 * after a fresh scan (flat), copied to *host_out.  Synchronises `stream`. */
per_status per_total(per_buffer *h, double *host_out, void *stream);

/* per_min -- the smallest p^alpha over filled slots: the root of the min tree (proportional) or
 * the minimum a fresh scan carries (flat); other modes are rejected.  Synchronises `stream`.
 * PER_ERR_EMPTY when no slot is filled. */
per_status per_min(per_buffer *h, float *host_out, void *stream);

/* per_size -- the number of filled slots as the host has counted the per_add calls enqueued
 * so far.  No device access.  Calls replayed from a CUDA graph are not counted here; the
 * device's own count is PER_STATE_COUNTERS[2] (per_read_state). */
per_status per_size(const per_buffer *h, uint64_t *out);

/* per_status_device -- read and clear the device error word (PER_DEVFLAG_* bits) into
 * *host_flags (may be NULL).  Synchronises `stream`.  Returns PER_ERR_DEVICE_FLAG when the
 * word was non-zero, PER_OK otherwise. */
per_status per_status_device(per_buffer *h, uint32_t *host_flags, void *stream);

/* per_last_error -- a description of the last failure on this handle ("" if none).  The
 * string stays valid until the next call on the handle.  NULL handle: the last per_create
 * failure on this thread. */
const char *per_last_error(const per_buffer *h);

/* What per_read_state copies out. */
enum {
    PER_STATE_LEAVES = 0,   /* float [nleaves]: p^alpha, 0 for empty slots (proportional) */
    PER_STATE_SUMS = 1,     /* double [nleaves]: internal sums, entry 0 unused */
    PER_STATE_MINS = 2,     /* float [nleaves]: internal mins, entry 0 unused */
    PER_STATE_RAW = 3,      /* float [capacity]: raw priorities (rank mode) */
    PER_STATE_CDF = 4,      /* double [capacity + 1]: rank CDF, entry 0 = 0 (rank mode) */
    PER_STATE_STATES = 5,   /* float [capacity x state_dim]: ring states */
    PER_STATE_NEXT = 6,     /* float [capacity x state_dim]: ring next_states */
    PER_STATE_ACTIONS = 7,  /* uint32 [capacity] */
    PER_STATE_REWARDS = 8,  /* float [capacity] */
    PER_STATE_DONES = 9,    /* uint8 [capacity] */
    PER_STATE_COUNTERS = 10, /* uint64 [5]: sample calls, cursor, size, max raw (float bits), and
                                (proportional mode) the latest update's crowding report:
                                bits 28-31 P, bits 20-27 a sequence number, bits 0-19 the
                                most entries one of its 2^P subtrees received (see
                                per_update_priorities) */
    PER_STATE_RANK_ORDER = 11, /* uint32 [size at the last sample]: slots by rank (rank mode) */
    PER_STATE_CUMULATIVE = 12  /* double [size on the device]: C[i] = leaves 0..i summed, as of the
                                  last sample, per_total or per_min (flat mode) */
};

/* per_read_state -- copy `count` elements starting at element `first` of one of the arrays
 * above into host memory at host_dst (inspection, checkpoints, tests).  Synchronises
 * `stream`.  PER_ERR_INVALID_ARG if the array does not exist in this mode or the range is
 * out of bounds. */
per_status per_read_state(per_buffer *h, uint32_t which, uint64_t first, uint64_t count,
                          void *host_dst, void *stream);

/* per_nleaves -- the tree's leaf count (power of two >= capacity). */
per_status per_nleaves(const per_buffer *h, uint64_t *out);

/*
 * per_rank_order_noalloc -- the slot order of the rank-based variant without a replay
 * buffer and without allocating: d_order[r-1] receives the slot of rank r, where rank 1 holds
 * the largest of d_raw[0, n) and equal priorities keep ascending slot order.  It runs the
 * same radix-sort kernels that per_sample uses in rank mode.  The pages have no counterpart:
 * this call exists for callers that may not allocate device memory -- code enqueuing work
 * while a CUDA graph is being captured (cudaMalloc is not permitted then), real-time loops
 * that forbid allocator latency, or hosts whose device memory belongs to another framework's
 * pool.  The call itself makes no cudaMalloc, cudaFree or other allocating call.
 *   d_raw    [n] float, device, > 0 and finite (caller-owned input).
 *   d_order  [n] uint32, device (caller-owned output).
 *   d_status one uint32, device, or NULL (caller-owned output): receives 0, or the
 *            PER_DEVFLAG_* bits of what the device met (PER_DEVFLAG_TIMEOUT: a bounded wait of
 *            the sort gave up).  The call returns before the GPU runs it, so its return value
 *            cannot carry this; read the word after the stream has reached it.
 *   n        1 .. 262144 (2^18); larger n returns PER_ERR_INVALID_ARG.
 * When a wait gave up, every entry of d_order is 0xFFFFFFFF (a value no valid slot has)
 * instead of a partial order, whether or not d_status is given.
 * Scratch: a fixed device array of about 4.3 MiB compiled into the library, which every GPU
 * that loads the library holds until the process exits.  The first call on a device looks up
 * that array's device address (cudaGetSymbolAddress) and caches it; make that first call on
 * each device before any stream capture begins.  All calls share the one array and it keeps
 * the last call's contents; every call first clears, with cudaMemsetAsync (no allocation), the
 * digit histograms, tile counters and error word that must start at zero, so a call that
 * stopped part way does not spoil the next.  Calls whose GPU work overlaps -- on different
 * streams, or concurrently from several host threads -- race on the array and must be
 * serialised by the caller.
 * Errors: PER_ERR_INVALID_ARG (NULL or misaligned pointer, n out of range), PER_ERR_CUDA.
 * It records no message for per_last_error.
 */
per_status per_rank_order_noalloc(const float *d_raw, uint32_t n, uint32_t *d_order,
                                  uint32_t *d_status, void *stream);

/* ---------------------------------------------------------------------------------------------
 * The learner's and the actor's operators beside the buffer: a loss per sampled row whose values
 * are the next priorities (distillation from a teacher's top logits), the recurrence of a
 * sequence model with its gradient, the verification of drafted tokens by an actor, and a paged
 * cache of keys and values with the attention of drafted trees over it.
 * They need no handle and keep nothing between calls: the caller owns every array, no call
 * allocates, and each enqueues one kernel (or copy; per_tree_attention one or two) on `stream`.  A failed call's message is
 * per_last_op_error(), on the calling thread.  Strides count elements; the innermost axis of
 * every array is contiguous.  Input strides may be any value (0 repeats a row for all); rows of an
 * output must not overlap.  Pointers need the alignment of their element type only; rows whose
 * start and stride are multiples of 16 bytes move in 16-byte pieces.  Others take longer on a GB300: a
 * recurrence with one such array (an odd number of channels, a shifted view) 1.4 to 2.4 times, a
 * verification of 512 rows of 131071 1.3 times.  Where d_status is given, a call sets PER_DEVFLAG_*
 * bits in it (it never clears them).
 * ------------------------------------------------------------------------------------------- */

/* per_last_op_error -- a description of the last failure of an operator on this thread ("" if none).
 * The string stays valid until the next failure on the thread. */
const char *per_last_op_error(void);

/* Element types of the operators' arrays.  Sums, normalisers, states and losses are float. */
enum { PER_TYPE_F32 = 0, PER_TYPE_F16 = 1, PER_TYPE_BF16 = 2 };

enum { PER_DISTILL_IDX64 = 1u };   /* per_distill_shape.flags: d_idx is int64, else int32 */

typedef struct {
    uint64_t rows;         /* N, 0 .. 2^31 - 1 (0 is a no-op) */
    uint32_t vocab;        /* V, 1 .. 2^18 */
    uint32_t top;          /* K, entries a teacher row has, 1 .. 1024 */
    uint32_t type;         /* PER_TYPE_* of the logits and of their gradient */
    uint32_t top_type;     /* PER_TYPE_* of the teacher's logits */
    int64_t stride_logits, stride_top, stride_idx, stride_grad;   /* between rows */
    float temperature;     /* tau, > 0 */
    uint32_t flags;        /* PER_DISTILL_* */
} per_distill_shape;

/*
 * per_distill_forward -- the loss of each row of student logits x against a teacher's top K
 * logits t at the places idx.  With lse_n = tau log sum_j exp(x_nj / tau) (over all V),
 * p_nj = exp((x_nj - lse_n) / tau) and q_nk = exp((t_nk - L_n) / tau):
 *     loss_n = tau^2 sum_k q_nk (log q_nk - log p_n,idx_nk).
 * L_n is the same soft maximum of the row's own teacher entries (their q sum to 1) or, where
 * d_teacher_lse is given, d_teacher_lse[n]: the teacher's over its whole vocabulary (q then sums to
 * the share that the top K hold).  An entry with idx < 0 is left out, whatever its t; one with
 * idx >= V is left out and sets PER_DEVFLAG_BAD_INDEX.  Entries that name one place several times
 * each count.  A row with no entry of q > 0, or whose logits are all -inf or at or below -2^100 (masked by the
 * lowest value of their type), has nothing to learn from: its loss and its gradient are 0.  A q > 0 where x is -inf gives a loss of +inf; NaN in x
 * or in a kept t gives NaN in its row.  The loss is not weighted: it is the row's next TD error
 * (per_update_priorities).
 *   d_logits [N x V], d_top [N x K], d_idx [N x K], d_teacher_lse [N] float or NULL,
 *   d_loss [N] float, d_lse [N] float (NULL to skip).
 * per_distill_backward -- its gradient from the saved d_lse, for row factors s (d_scale [N] float;
 * NULL: 1), an importance weight over the batch's size or what an outer gradient brings:
 *     grad_nj = s_n tau (S_n p_nj - sum over k with idx_nk = j of q_nk),  S_n = sum_k q_nk.
 * per_distill_step -- loss, lse and gradient in one pass over the logits (read once, gradient
 * written once; a row stays in the shared memory of up to 8 CTAs: 1, 2, 4 or 8 so that a part takes at most
 * 64 KB, or 8 of larger parts.  A vocabulary just past 2^15, 2^16 or 2^17 16-bit elements or half as many of 32 bits
 * is in parts of half the size and takes 1.4 to 1.75 times as long per byte on a GB300; float rows of 2^18 take twice
 * as long per byte as those of 2^17).
 * d_grad may be d_logits itself (same stride): the gradient then takes the logits' place.
 * The gradient is rounded once to its type.  Before that, with U = 2^-24 and y = (x - lse) / tau, a p is good to a
 * relative 9 U + |y| U (the rounding of x - lse) for float logits and 9 U + 2 |y| U for 16-bit ones, beside what lse's
 * own error brings (tau U (ln V + 32), and |lse| U); a p below 2^-126 counts as 0.  Losses take their differences
 * from the rows' largest entries, so that what all logits of a row share costs them no digits.  Results do not depend
 * on the launch's order.
 */
per_status per_distill_forward(const per_distill_shape *shape, const void *d_logits, const void *d_top,
                               const void *d_idx, const float *d_teacher_lse, float *d_loss,
                               float *d_lse, uint32_t *d_status, void *stream);
per_status per_distill_backward(const per_distill_shape *shape, const void *d_logits, const void *d_top,
                                const void *d_idx, const float *d_teacher_lse, const float *d_lse,
                                const float *d_scale, void *d_grad, uint32_t *d_status, void *stream);
per_status per_distill_step(const per_distill_shape *shape, const void *d_logits, const void *d_top,
                            const void *d_idx, const float *d_teacher_lse, const float *d_scale,
                            float *d_loss, float *d_lse, void *d_grad, uint32_t *d_status,
                            void *stream);

enum { PER_VERIFY_TOKENS64 = 1u };   /* per_verify_shape.flags: d_tokens is int64, else int32 */

typedef struct {
    uint32_t batch;        /* B, 0 .. 2^20 (0 is a no-op) */
    uint32_t drafts;       /* D, drafted tokens a sequence has at most, 0 .. 1024 */
    uint32_t vocab;        /* V, 1 .. 2^18 */
    uint32_t type;         /* PER_TYPE_* of the probabilities */
    int64_t stride_p[2], stride_q[2];      /* between sequences, between positions */
    int64_t stride_tokens, stride_u;       /* between sequences */
    uint32_t flags;        /* PER_VERIFY_* */
    uint32_t reserved;     /* 0 */
} per_verify_shape;

/*
 * per_verify_draft -- verify drafted tokens against the target's probabilities so that what is
 * emitted follows the target's distribution.  Sequence b drafted m = d_lens[b] tokens (clamped to
 * 0 .. D; D where d_lens is NULL).  Token i is accepted when every one before it was and
 *     u_i q_i(token_i) < p_i(token_i)      (the product rounded to binary32),
 * with p_i row i of d_p, q_i row i of d_q, or q = 1 where d_q is NULL (a draft that was certain of its
 * token).  With n the number accepted, one more token is drawn: after a refusal (n < m) from the
 * masses max(p_n(j) - q_n(j), 0) (binary32; with d_q NULL p_n without token_n), else from p_m.  The draw is exact
 * in integers, so it does not depend on any order of summation: a mass counts floor(2^40 mass)
 * units (NaN and negative 0, above 1 as 1), M is their sum, and with U = floor(2^31 u) (u =
 * d_sample_u[b], held to 0 <= U < 2^31; NaN: 0) the token is the first j whose inclusive sum exceeds
 * floor(U M / 2^31).  M = 0 draws from p_n instead; if that holds nothing either, the token is -1.
 * D = 0 draws one token from each row of p.  A drafted token outside [0, V) has p = q = 0: it is
 * refused, and if the verification reaches it PER_DEVFLAG_BAD_INDEX is set.
 *   d_p [B x (D + 1) x V], d_q [B x D x V] or NULL, d_tokens [B x D], d_lens [B] int32 or NULL,
 *   d_accept_u [B x D] float, d_sample_u [B] float, d_accepted [B] int32 (n),
 *   d_out [B x (D + 1)] int32 (contiguous): the accepted tokens, the drawn one, then -1,
 *   d_accept_p [B x D] float (contiguous) or NULL: min(1, p_i / q_i) of every drafted token (1 where
 *   q_i <= p_i), 0 past m and for a token outside [0, V): what a buffer of drafts can take as its
 *   rows' priorities.
 */
per_status per_verify_draft(const per_verify_shape *shape, const void *d_p, const void *d_q,
                            const void *d_tokens, const int32_t *d_lens, const float *d_accept_u,
                            const float *d_sample_u, int32_t *d_accepted, int32_t *d_out,
                            float *d_accept_p, uint32_t *d_status, void *stream);

/* per_scan_shape.flags */
enum {
    PER_SCAN_SIGMOID = 1u,   /* a is a gate before its sigmoid; without it a is the decay itself */
    PER_SCAN_REVERSE = 2u    /* time runs from the last step to the first */
};

typedef struct {
    uint64_t steps;        /* T, 0 .. 2^31 - 1 */
    uint32_t batch;        /* B */
    uint32_t channels;     /* C; B C < 2^31 */
    uint32_t type;         /* PER_TYPE_* of a, x, h and their gradients */
    uint32_t flags;        /* PER_SCAN_* */
    int64_t stride_a[2], stride_x[2], stride_h[2];       /* between sequences, between steps */
    int64_t stride_gh[2], stride_ga[2], stride_gx[2];    /* the gradients' (per_scan_backward) */
    int64_t stride_resets[2];
    uint32_t *d_status;    /* device word or NULL: PER_DEVFLAG_TIMEOUT is set in it when a wait ran out */
    uint32_t wait_limit_ms; /* limit of a wait between the parts of a sequence, 0 .. 10000 (0: 2000) */
    uint32_t withhold;     /* 0.  To test the limit: the part, 1 .. 16, of each sequence split over parts
                              that tells the others nothing */
} per_scan_shape;

/*
 * per_scan_forward -- the gated linear recurrence over T steps, channel by channel:
 *     h_t = a_t h_{t-1} + x_t                        (decays given), or
 *     h_t = f_t h_{t-1} + (1 - f_t) x_t, f = 1 / (1 + exp(-a))      (PER_SCAN_SIGMOID).
 * h_{-1} is d_h0 (NULL: 0).  A step with d_resets[b, t] != 0 starts an episode: the state that comes into it counts
 * as 0, whatever it holds.  A weight of exactly 0 likewise drops what it multiplies, infinities and NaN
 * too (a gate of -inf drops the state, of +inf the input: padding can hold anything).  The
 * state is kept in binary32; h is rounded to its type where it is stored.  f and 1 - f are good to a
 * relative 2^-21 where a is binary32, to 2^-21 + |a| 2^-24 where it is not; an f or 1 - f below 2^-126 may
 * count as 0.  Long sequences are split over time where the channels alone do not fill the GPU; the
 * joints multiply the decays of a stretch, whose product must stay finite in binary32 (decays of
 * magnitude at most 1 always do; a product below 2^-126 is known to 2^-149, so that a state of size s
 * can be off by s 2^-149 behind it).  The parts of a split sequence wait for one another with a limit.
 * A wait that runs out sets PER_DEVFLAG_TIMEOUT in d_status; states that are then not known are NaN,
 * and so is what follows from them.  PER_SCAN_REVERSE runs t = T-1 .. 0 (discounted returns: a = gamma,
 * x = reward, a reset at each episode's last step).
 *   d_a, d_x [B x T x C], d_h0 [B x C] float or NULL, d_resets [B x T] uint8 or NULL,
 *   d_h [B x T x C], d_last [B x C] float (NULL to skip): the state after the last step; it may be
 *   d_h0 itself.  T = 1 is the step of a model that is being served.  T = 0 copies h0 to last.
 * per_scan_backward -- its gradients for d_gh (of h) and d_glast (of last; NULL: 0), reading the h that the
 * forward call stored.  With w_t the weight of h_{t-1} (0 at a reset) and g_t = gh_t + w_{t+1} g_{t+1}:
 *     ga_t = g_t h_{t-1}, gx_t = g_t                                       (decays given), or
 *     ga_t = g_t (h_{t-1} - x_t) f_t (1 - f_t), gx_t = g_t (1 - f_t)       (PER_SCAN_SIGMOID),
 *     gh0 = w_0 g_0.       (h_{t-1} counts as 0 at a reset.)
 *   d_x may be NULL where decays are given.  d_ga, d_gx [B x T x C] and d_gh0 [B x C] float, each may be
 *   NULL to skip.
 * Outputs must not overlap inputs except where said.
 */
per_status per_scan_forward(const per_scan_shape *shape, const void *d_a, const void *d_x,
                            const float *d_h0, const uint8_t *d_resets, void *d_h, float *d_last,
                            void *stream);
per_status per_scan_backward(const per_scan_shape *shape, const void *d_a, const void *d_x,
                             const void *d_h, const float *d_h0, const uint8_t *d_resets,
                             const void *d_gh, const float *d_glast, void *d_ga, void *d_gx,
                             float *d_gh0, void *stream);

/* ---------------------------------------------------------------------------------------------
 * Drafted trees over a paged cache: what an actor's target needs around per_verify_draft.  Keys and
 * values lie in pages of S slots; row b of a table names the pages of sequence b in order, so that its
 * slot s is slot s mod S of page table[b, s / S].  A sequence's first `start` (or `len`) slots hold its
 * context; a call's new tokens (the nodes of a tree, each one token) take the slots behind it in their order.
 * Nothing beyond a sequence's own slots is read into a result: what stale slots hold, NaN too, does not
 * matter.  A table entry outside [0, P), a slot behind the table's end, a negative start and a count that
 * is out of range set PER_DEVFLAG_BAD_INDEX; what they name is left out (not written, not attended to; a negative d_lens
 * counts as no context in per_tree_attention).  What is written to, keys and values, must not overlap (one and the same
 * memory is refused; attention may read both from one).
 * ------------------------------------------------------------------------------------------- */

typedef struct {
    uint32_t pages;        /* P, 0 .. 2^31 - 1 */
    uint32_t page;         /* S, slots of a page, 1 .. 2^20 */
    uint32_t width;        /* pages that a row of the table names; width S at most 2^30 */
    uint32_t heads;        /* Hkv, heads of keys and values, 1 .. 4096 */
    uint32_t dim;          /* D, entries of a head, 1 .. 256 */
    uint32_t type;         /* PER_TYPE_* of the cache and of all that goes in and out of it */
    int64_t stride_table;                  /* between sequences */
    int64_t stride_k[3], stride_v[3];      /* between pages, slots of a page, heads (any layout) */
} per_cache;

enum { PER_APPEND_INTERLEAVED = 1u };   /* per_append_shape.flags: entries 2 j and 2 j + 1 turn together, else j and j + rot / 2 */

typedef struct {
    per_cache cache;
    uint32_t batch;        /* B, 0 .. 2^20 (0 is a no-op) */
    uint32_t tokens;       /* N, new tokens a sequence has at most; B N < 2^31 (0 is a no-op) */
    uint32_t q_heads;      /* Hq, heads of queries, 0 .. 4096 (0: no queries) */
    uint32_t rot;          /* entries of a head that are rotated, even, 0 .. D */
    int64_t stride_in[2][3];               /* of k and of v: between sequences, tokens, heads */
    int64_t stride_q[3], stride_q_out[3];
    int64_t stride_positions;              /* between sequences */
    uint32_t flags;        /* PER_APPEND_* */
    uint32_t reserved;     /* 0 */
} per_append_shape;

/*
 * per_cache_append -- keys and values of new tokens into their slots, keys and queries rotated by their
 * positions on the way.  Token i < d_counts[b] of sequence b goes to slot d_starts[b] + i.  With pos =
 * d_positions[b, i] (NULL: d_starts[b] + i) and theta_j = pos d_inv_freq[j], for j < rot / 2,
 *     x'_j = x_j cos theta_j - x_j* sin theta_j,    x'_j* = x_j* cos theta_j + x_j sin theta_j,
 * where j* = j + rot / 2 (or the places are 2 j and 2 j + 1 with PER_APPEND_INTERLEAVED); entries from
 * rot on, and values, are copied as they are.  The angle is reduced in 64-bit fixed point: theta is off by
 * at most 2^-23 of a radian for any 32-bit position and |d_inv_freq| <= 1.  Sums are binary32, rounded once.
 * Queries need no cache: they are rotated into d_q_out (which may be d_q itself, same strides);
 * those of tokens i >= d_counts[b] come out as 0.  Nothing else is written: slots outside
 * [start, start + count) keep what they hold.  Two tokens must not name one slot of one page.
 *   d_k, d_v [B x N x Hkv x D], d_q, d_q_out [B x N x Hq x D] (NULL where Hq is 0), d_table [B x width]
 *   int32, d_starts [B] int32, d_counts [B] int32 or NULL (N), d_positions [B x N] int32 or NULL,
 *   d_inv_freq [rot / 2] float (NULL where rot is 0).
 */
per_status per_cache_append(const per_append_shape *shape, const void *d_k, const void *d_v, const void *d_q,
                            void *d_k_cache, void *d_v_cache, void *d_q_out, const int32_t *d_table,
                            const int32_t *d_starts, const int32_t *d_counts, const int32_t *d_positions,
                            const float *d_inv_freq, uint32_t *d_status, void *stream);

typedef struct {
    per_cache cache;
    uint32_t batch;        /* B, 0 .. 2^20 (0 is a no-op) */
    uint32_t nodes;        /* N, nodes a sequence has at most, 0 .. 1024 (0 is a no-op) */
    uint32_t q_heads;      /* Hq, a multiple of Hkv, at most 64 to each: query head h reads head h / (Hq / Hkv) */
    float scale;           /* of the scores, finite */
    int64_t stride_q[3], stride_out[3];    /* between sequences, nodes, heads */
    int64_t stride_mask[2];                /* between sequences (0: one mask for all), between nodes */
    uint64_t work_bytes;   /* of d_work */
    uint32_t wait_limit_ms; /* limit of a wait inside the kernel, 0 .. 10000 (0: 2000) */
    uint32_t withhold;     /* 0.  To test the limit: the barrier, 1 .. 8, that waits for an arrival which never comes: of keys, of
                              values, of a tile's release, of the warps among one another; with many rows also of queries, of
                              scores, of p, of outputs (a kernel that has no such barrier runs as with 0) */
} per_attend_shape;

/*
 * per_tree_attention -- attention of the drafted nodes of each sequence over its context and over one
 * another.  Node i < m = d_counts[b] of sequence b sees the d_lens[b] tokens of the context and those nodes j < m,
 * in slots d_lens[b] + j, that its mask names (d_mask[b, i, j] != 0; NULL: j <= i, a chain).  Over what it sees,
 *     out_i = sum_j p_ij v_j,   p_ij = exp(s_ij - lse_i),   s_ij = scale q_i . k_j,   lse_i = log sum_j exp s_ij.
 * A node that sees nothing (or only scores of -inf) gives 0 and an lse of -inf, and so does a node
 * i >= m.  What a node does not see takes no part, whatever it holds (infinities and NaN too).  N = 1
 * is the step of plain decoding.  Products of 16-bit types are summed in binary32, scores and their
 * sums are binary32, and p is rounded once to the type before its product with v (the sum of p is
 * not; as float16, a p below 2^-25 of its row's largest is off by up to 2^-36 of that), or, with up to 16 rows (nodes times
 * query heads) to a head of keys on 16-byte boundaries, taken in two rounded parts.  binary32 entries are
 * taken as two parts whose products give 21 bits.  Out is rounded once.
 * Scores may be as large as binary32 holds (times log2(e)); what is past that is infinite.  Sums of p v are divided by the sum
 * of p at the end: they, with p of up to 2^8, must be within binary32 (|v| below 2^120 over the number of keys, say).
 *   d_q, d_out [B x N x Hq x D] (not the same memory), d_mask [B x N x N] bytes, d_lens, d_counts [B] int32 (counts NULL: N),
 *   d_table [B x width] int32, d_lse [B x N x Hq] float (contiguous) or NULL, d_work: work_bytes of scratch
 *   memory (16-byte aligned) that this call alone uses until it has run; per_tree_attention_work says
 *   how much.
 * Which CTA takes which part depends on the lengths alone, and parts are joined in their order: the same
 * inputs give the same bits.  A value that is not finite gives NaN or infinity in the rows that see it.  Caches whose
 * heads begin on 16 bytes and whose axes lie in one another (each stride a multiple of the next smaller one) are copied by
 * tiles; others entry by entry, several times slower.  Waits inside the kernel have a limit, after which the kernel waits
 * for its copies and products under way (with the same limit for each), sets PER_DEVFLAG_TIMEOUT and ends; results are not valid.
 * per_tree_attention_work -- the bytes of d_work that a call of this shape with these caches needs on the current
 * device (which kernel takes it depends on where they lie; nothing is read).
 */
per_status per_tree_attention(const per_attend_shape *shape, const void *d_q, const void *d_k_cache,
                              const void *d_v_cache, const int32_t *d_table, const int32_t *d_lens,
                              const int32_t *d_counts, const uint8_t *d_mask, void *d_out, float *d_lse,
                              void *d_work, uint32_t *d_status, void *stream);
per_status per_tree_attention_work(const per_attend_shape *shape, const void *d_k_cache, const void *d_v_cache,
                                   uint64_t *bytes);

typedef struct {
    per_cache cache;
    uint32_t batch;        /* B, 0 .. 2^20 (0 is a no-op) */
    uint32_t nodes;        /* N, nodes of a tree, 0 .. 2^20 */
    uint32_t most;         /* L, entries that a path has at most, 0 .. 1024 (0 is a no-op) */
    uint32_t reserved;     /* 0 */
    int64_t stride_path;   /* between sequences */
} per_keep_shape;

/*
 * per_cache_keep -- the accepted path of each tree moved to where its sequence goes on: for j <
 * d_kept[b], keys and values of slot d_lens[b] + d_path[b, j] go to slot d_lens[b] + j.  A path goes from node to
 * later node: 0 <= path_0 < path_1 < ... < N.  The first entry that breaks this (or lies in a page
 * that does not exist) ends the path: it and what follows stay, and PER_DEVFLAG_BAD_INDEX is set.  The caller
 * then counts d_kept[b] more tokens of context.  A page must not lie in two rows of the table if a move
 * writes to it.
 *   d_table [B x width] int32, d_lens [B] int32, d_path [B x L] int32, d_kept [B] int32 (0 .. L).
 */
per_status per_cache_keep(const per_keep_shape *shape, void *d_k_cache, void *d_v_cache, const int32_t *d_table,
                          const int32_t *d_lens, const int32_t *d_path, const int32_t *d_kept, uint32_t *d_status,
                          void *stream);

#ifdef __cplusplus
}
#endif
#endif
