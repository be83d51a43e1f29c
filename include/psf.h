/*
 * psf.h -- C ABI of the packed-sequence flash-attention library (libpsf.so).
 *
 * Exact softmax attention over packed variable-length sequences on one GB300
 * (sm_103a): forward returning out and an fp32 log-sum-exp, backward from
 * caller-supplied out/lse returning dQ and dK/dV reduced to the KV heads, and
 * the doc-ids -> varlen-segment builder that feeds them.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Pointers are DEVICE pointers owned by the caller; the library allocates
 *    nothing. Outputs and workspaces are caller-allocated. Tensor base pointers
 *    must be 16-byte aligned (a TMA requirement).
 *  - Strides: the attention calls take `strides`, NULL for the layout's
 *    contiguous strides, else an int64 array of element strides, three per
 *    tensor in the order (batch, head, row), tensors in the order each call
 *    lists. The head dim is always contiguous. A stride of a dimension of
 *    extent 1 (the batch of a packed THD tensor, a single head or row) is
 *    ignored; every other one must be a positive multiple of 8 elements
 *    (16 bytes) below 2^38, and an output's strides must not make it overlap
 *    itself (PSF_EINVAL otherwise). lse stays contiguous.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *    Every call is asynchronous on that stream.
 *  - Return value: PSF_OK (0) after a successful launch, or a negative code.
 *    No exception crosses the ABI. psf_last_error() gives a message for the
 *    last failing call on the calling thread.
 *  - Kernel-side faults in the caller's data (bad segment arrays) and pipeline
 *    waits that ran out are recorded in a per-device status word that
 *    psf_device_status() returns after synchronising the device.
 *  - dtype: bf16 or fp16 inputs and outputs (`out`, `dq`, `dk`, `dv`), chosen
 *    per call by a PSF_DTYPE_* argument; lse and the row-dot Delta are fp32.
 *  - Head dims (Dqk, Dv) supported: (64,64), (128,128), (192,128), (512,512).
 *    The (512,512) backward launches four-CTA thread-block clusters, as many
 *    as the device holds at once; where it holds none (PSF_ECUDA).
 *  - GQA: Hq % Hkv == 0; query head h uses KV head h / (Hq / Hkv).
 *  - Causal masks are aligned to the bottom-right corner of each segment
 *    (dense: of the Nq x Nk matrix): local query i of a segment with m queries
 *    and n keys sees local key j iff j <= i + (n - m).
 *  - window_left > 0 is a left window that counts the current token: key j is
 *    visible only if j >= i + (n - m) - window_left + 1. window_left < 0 (for
 *    example INT32_MIN, the pages' "no window" sentinel) means unbounded;
 *    window_left == 0 is rejected with PSF_EINVAL.
 *  - Query rows covered by no segment, and rows that see no key, get out = 0
 *    and lse = -inf; the backward treats lse = -inf as zero probability.
 *  - scale must be finite and > 0.
 */
#ifndef PSF_H_
#define PSF_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PSF_OK 0
#define PSF_EINVAL (-1)        /* bad argument: shape, null pointer, alignment, window == 0, scale */
#define PSF_EUNSUPPORTED (-2)  /* no kernel for this head-dim pair, or the device is not sm_103 */
#define PSF_ECUDA (-3)         /* a CUDA runtime call (launch, tensor-map encode) failed */
#define PSF_EDEVICE_ARGS (-4)  /* kernel-side validation rejected the segment arrays */
#define PSF_ETIMEOUT (-5)      /* a pipeline wait inside a kernel exceeded its limit */
#define PSF_EWORKSPACE (-6)    /* workspace pointer null or smaller than the size query */

/* Tensor layouts accepted by the varlen calls. */
#define PSF_LAYOUT_THD 0  /* packed [T, H, D]; lse [H, T]                                */
#define PSF_LAYOUT_BHSD 1 /* batched [B, H, S, D]; lse [B, H, S]; rows are b * S + s     */

/*
 * Element type of the 16-bit tensors of a call (q, k, v, out, dout, dq, dk, dv,
 * merge operands); one type per call. lse, Delta and every accumulator stay
 * fp32.                     [ffpa_attention page, module docstring: the op
 *                            takes bf16 and fp16 inputs]
 */
#define PSF_DTYPE_BF16 0
#define PSF_DTYPE_F16 1

/* Message for the last failing call on this thread (never NULL). */
const char* psf_last_error(void);

/* 1 if the current device is an sm_103 GPU this library was built for, else 0. */
int psf_device_supported(void);

/*
 * Synchronise the current device and return the first kernel-side status
 * recorded since the last clear: PSF_OK, PSF_EDEVICE_ARGS or PSF_ETIMEOUT.
 * clear != 0 resets it to PSF_OK.
 */
int psf_device_status(int clear);

/* Upper bound, in nanoseconds, of every pipeline wait inside the kernels
 * (default 2e9, or $PSF_WAIT_LIMIT_NS when set at load time). A kernel that gives
 * up still waits for its own copies and products under way, 1e8 at least. */
void psf_set_wait_limit_ns(uint64_t ns);

/*
 * Check of the failure path every pipeline wait takes, without a fault: one
 * CTA of 64 threads on `stream` whose warp 0 waits on an mbarrier that expects
 * one arrival. With arrive != 0 warp 1 arrives and the kernel ends at once;
 * with arrive == 0 nothing arrives, the wait gives up after the current wait
 * limit (psf_set_wait_limit_ns), records PSF_ETIMEOUT in the status word that
 * psf_device_status() reads, and the kernel returns normally, leaving the
 * context usable. Returns PSF_OK once launched (PSF_EUNSUPPORTED on another
 * device, PSF_ECUDA if the launch fails).
 */
int psf_check_pipeline_wait(int arrive, void* stream);

/*
 * Kernel timing for profiling. psf_kernel_timing(1) clears the record and
 * starts it: from then on every attention call records two CUDA events on its
 * stream, immediately before and after its main kernel (kind 0: forward main
 * kernel, kind 1: backward main kernel). psf_kernel_timing(0) stops recording.
 * psf_kernel_times_ms() waits for the recorded events of `kind` and returns
 * their summed device time in *total_ms and their number in *launches.
 * Calls made while a stream capture is active record the pair as event-record
 * nodes of the captured graph: each replay of the graph re-records them, and
 * psf_kernel_times_ms() after a replay returns that replay's kernel times.
 */
int psf_kernel_timing(int enable);
int psf_kernel_times_ms(int kind, double* total_ms, int* launches);

/*
 * Workspace sizes in bytes. total_q_rows / total_k_rows count the flattened
 * query / key rows (T for THD, B * S for BHSD); nseg is the number of segments
 * (or the capacity passed to the builder).
 */
size_t psf_attn_fwd_workspace_size(int64_t total_q_rows, int nseg);
size_t psf_attn_bwd_workspace_size(int64_t total_q_rows, int64_t total_k_rows, int nseg, int Hq, int Hkv, int Dqk,
                                   int Dv);

/*
 * Varlen forward.           [ffpa_attention page, `_ffpa_varlen_fwd`: packed THD
 *                            inputs, cu_q/cu_k/max_q/max_k/scale/causal, returns
 *                            (out[T,Hq,D], lse[Hq,T]); left window per the
 *                            attention utils page, `window_size`]
 *  q [Tq,Hq,Dqk], k [Tk,Hkv,Dqk], v [Tk,Hkv,Dv] -> out [Tq,Hq,Dv], lse [Hq,Tq]
 *  (layout PSF_LAYOUT_THD), or the BHSD forms with Tq = B*Sq, Tk = B*Sk and
 *  lse [B,Hq,Sq] (layout PSF_LAYOUT_BHSD; a segment must not cross a batch row).
 *  cu_q / cu_k: int32 [nseg+1] device arrays of exclusive prefix sums over the
 *  flattened rows; segment s pairs queries [cu_q[s], cu_q[s+1]) with keys
 *  [cu_k[s], cu_k[s+1]); zero-length segments are allowed.
 *  dev_meta: nullable int32[3] device array {nseg, max_q, max_k} written by
 *  psf_build_doc_segments; when given, the segment count and maxima are read
 *  from it on the device and `nseg` is only the capacity of cu_q/cu_k.
 *  max_q / max_k: the longest segment lengths (ignored when dev_meta is given);
 *  a longer segment is a PSF_EDEVICE_ARGS device status.
 *  softcap: 0 (off), or c > 0: every logit z = scale * q . k becomes
 *  c * tanh(z / c) before the mask and the softmax (lse is over the capped
 *  logits). Negative or non-finite values are PSF_EINVAL.
 *                           [ffpa_attention page, `ffpa_attention_forward`
 *                            softcap argument; the eager attention the page
 *                            falls back to for it caps the scaled scores so]
 *  flags: 0, or PSF_FWD_PACK_GQA: the G = Hq / Hkv query heads of a KV head
 *  share one 128-row tile (128 / G rows of each), so short segments fill the
 *  tile and K/V are loaded once for all G heads. Same results; it applies to
 *  head dims (64, 64) and (128, 128) with G in 2..16 dividing 128, and other
 *  shapes run one head per tile.
 *                           [ffpa_attention page, `_ffpa_varlen_fwd`: the
 *                            pack-GQA sentinel the pages fix off]
 *  Any other bit is PSF_EINVAL.
 *  strides: NULL, or 12 element strides (batch, head, row) of q, k, v, out;
 *  for THD the row stride steps tokens and the batch stride is ignored.
 *  workspace: psf_attn_fwd_workspace_size(Tq, nseg) bytes (enough for either flag).
 */
#define PSF_FWD_PACK_GQA 1
int psf_attn_varlen_fwd(const void* q, const void* k, const void* v, void* out, float* lse, const int32_t* cu_q,
                        const int32_t* cu_k, const int32_t* dev_meta, int nseg, int max_q, int max_k, int layout,
                        int dtype, int B, int Sq, int Sk, int Hq, int Hkv, int Dqk, int Dv, const int64_t* strides,
                        float scale, int causal, int32_t window_left, float softcap, int flags, void* workspace,
                        size_t ws_bytes, void* stream);

/*
 * Varlen forward that allocates nothing and takes no workspace.
 *                           [no counterpart on the pages: an addition of this
 *                            library for callers that cannot allocate]
 *  Some callers cannot call cudaMalloc on this path: runtimes that reserve all
 *  device memory up front and hand out nothing afterwards, plugin hosts that
 *  own every allocation, or code that must not touch the allocator while a
 *  step runs. This entry point behaves like psf_attn_varlen_fwd (same
 *  arguments minus strides, softcap, flags, workspace and ws_bytes: contiguous
 *  tensors, no softcap, one query head per tile, same results) but keeps its tile
 *  schedule in a fixed array in the library's device memory (852,736 bytes,
 *  held on every GPU that loads the library until the process exits).
 *  Limits: B * Sq <= PSF_NOALLOC_MAX_Q_ROWS and nseg <= PSF_NOALLOC_MAX_SEGMENTS;
 *  larger calls return PSF_EINVAL without launching anything.
 *  The first call on a device looks up that array's device address (with the
 *  device current); make that first call before any stream capture.
 *  Every call shares the one array and leaves its contents behind; the
 *  schedule kernel rewrites all of it that a call reads, so nothing needs
 *  clearing between calls. Calls whose kernels overlap on the GPU (different
 *  streams, or different host threads, without ordering between them) race on
 *  the array and must not be issued.
 */
#define PSF_NOALLOC_MAX_Q_ROWS (1 << 20)
#define PSF_NOALLOC_MAX_SEGMENTS 65536
int psf_attn_varlen_fwd_noalloc(const void* q, const void* k, const void* v, void* out, float* lse,
                                const int32_t* cu_q, const int32_t* cu_k, const int32_t* dev_meta, int nseg,
                                int max_q, int max_k, int layout, int dtype, int B, int Sq, int Sk, int Hq, int Hkv,
                                int Dqk, int Dv, float scale, int causal, int32_t window_left, void* stream);

/*
 * Varlen backward from caller-supplied out / lse.
 *                           [ffpa_attention page, `_ffpa_varlen_bwd`: "using the
 *                            caller-supplied out/lse. Returns (dq, dk, dv)"]
 *  Same layouts and segment rules as the forward. dout has the layout of out.
 *  dq has q's layout; dk / dv have k's / v's layout (Hkv heads: the gradients of
 *  the Hq / Hkv query heads sharing a KV head are summed on chip).
 *  Keys that no query sees get dk = dv = 0; query rows outside every segment
 *  get dq = 0.
 *  softcap: the forward's (0 = off); with c > 0, dS carries 1 - tanh^2(z / c).
 *  flags: 0, or PSF_BWD_PACK_GQA: each step takes the G = Hq / Hkv query heads
 *  of its KV head, 128 / G rows each (head dims up to 128 with G = 2 or 4 and
 *  no softcap; other calls take one head per step). Same results; for short segments,
 *  where one head's rows fill little of a 128-row step. Other bits: PSF_EINVAL.
 *  strides: NULL, or 24 element strides (batch, head, row) of q, k, v, out,
 *  dout, dq, dk, dv.
 *  workspace: psf_attn_bwd_workspace_size(Tq, Tk, nseg, Hq, Hkv, Dqk, Dv) bytes
 *  (holds the fp32 dQ accumulator, Delta = rowsum(dO * out), the tile schedule
 *  and, for head dims up to 128, the fp32 dK/dV partial sums of key tiles cut
 *  across SMs; its size grows with Tq, not with Tk beyond the schedule).
 */
int psf_attn_varlen_bwd(const void* dout, const void* q, const void* k, const void* v, const void* out,
                        const float* lse, void* dq, void* dk, void* dv, const int32_t* cu_q, const int32_t* cu_k,
                        const int32_t* dev_meta, int nseg, int max_q, int max_k, int layout, int dtype, int B, int Sq,
                        int Sk, int Hq, int Hkv, int Dqk, int Dv, const int64_t* strides, float scale, int causal,
                        int32_t window_left, float softcap, int flags, void* workspace, size_t ws_bytes,
                        void* stream);
#define PSF_BWD_PACK_GQA 1

/*
 * Dense forward on SDPA-layout tensors.
 *                           [ffpa_attention page, `_ffpa_dense_fwd`: [B,H,N,D]
 *                            inputs, returns (out[B,Hq,Nq,D], lse[B,Hq,Nq] fp32),
 *                            GQA and causal/non-causal handled internally;
 *                            fa4 page, `causal_fa4_attention`]
 *  q [B,Hq,Nq,Dqk], k [B,Hkv,Nk,Dqk], v [B,Hkv,Nk,Dv], out [B,Hq,Nq,Dv],
 *  lse [B,Hq,Nq]. Causal is bottom-right aligned when Nq != Nk.
 *  strides: NULL (contiguous [B,H,N,D]) or 12 element strides (batch, head,
 *  row) of q, k, v, out: for example a [B,N,H,D] tensor seen as [B,H,N,D]
 *  (strides N*H*D, D, H*D) is read in place.
 *  softcap, flags: as for psf_attn_varlen_fwd.
 *  workspace: psf_attn_fwd_workspace_size(B * Nq, B) bytes.
 */
int psf_attn_dense_fwd(const void* q, const void* k, const void* v, void* out, float* lse, int B, int Hq, int Hkv,
                       int Nq, int Nk, int Dqk, int Dv, const int64_t* strides, int dtype, float scale, int causal,
                       int32_t window_left, float softcap, int flags, void* workspace, size_t ws_bytes,
                       void* stream);

/*
 * Dense backward.           [ffpa_attention page, `_ffpa_dense_bwd`: returns
 *                            (dq, dk, dv) in [B,H,N,D], dK/dV reduced to Hkv]
 *  strides: NULL or 24 element strides (batch, head, row) of q, k, v, out,
 *  dout, dq, dk, dv.
 *  softcap, flags: as for psf_attn_varlen_bwd.
 *  workspace: psf_attn_bwd_workspace_size(B * Nq, B * Nk, B, Hq, Hkv, Dqk, Dv) bytes.
 */
int psf_attn_dense_bwd(const void* dout, const void* q, const void* k, const void* v, const void* out,
                       const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int Nq, int Nk,
                       int Dqk, int Dv, const int64_t* strides, int dtype, float scale, int causal,
                       int32_t window_left, float softcap, int flags, void* workspace, size_t ws_bytes,
                       void* stream);

/*
 * Doc ids -> varlen segments, on the GPU.
 *                           [fa4 page, module docstring bullets 1-3,
 *                            `_varlen_segments`, `_varlen_layout`]
 *  kv_doc_ids: int32 [B, Sk] document ids (1-based, 0 = padding) of all keys.
 *  The local query shard is [q_global_start, q_global_start + q_length) of
 *  every row. Every maximal run of equal id (padding runs included) is split at
 *  the end of the shard; each piece contributes its overlap with the shard as
 *  queries and all of its tokens as keys; pieces without queries become
 *  zero-query segments, so the key segments tile the flattened [B * Sk] rows
 *  and the query segments tile [B * q_length]. Segments are listed row-major.
 *  Outputs: cu_q, cu_k (int32, capacity + 1 entries each, prefix sums),
 *  dev_meta int32[3] = {nseg, max_q, max_k}, and seg_is_pad (nullable, uint8
 *  [capacity]: 1 for a segment cut from a padding run).
 *  flags: 0, or PSF_SEGMENTS_SKIP_PAD: every piece cut from a padding run is
 *  written as two segments, its queries with no keys, then its keys with no
 *  queries. The attention then gives padding queries out = 0 and lse = -inf by
 *  itself (no psf_pad_fixup needed) and computes no padding-vs-padding pairs;
 *  dK/dV of padding keys come out 0. Any other bit is PSF_EINVAL.
 *                           [fa4 page, `document_causal_fa4_attention`: padding
 *                            queries are zero; cp_attention page,
 *                            `_build_packed_ring_segments`: pad query rows zeroed]
 *  capacity: room in cu_q / cu_k; B * Sk + B always suffices without flags,
 *  2 * (B * Sk + B) with PSF_SEGMENTS_SKIP_PAD. Too small a capacity is a
 *  PSF_EDEVICE_ARGS device status (dev_meta[0] is then 0).
 *  Requires 0 <= q_global_start, q_global_start + q_length <= Sk.
 */
#define PSF_SEGMENTS_SKIP_PAD 1
int psf_build_doc_segments(const int32_t* kv_doc_ids, int B, int Sk, int q_length, int q_global_start,
                           int32_t* cu_q, int32_t* cu_k, int capacity, int32_t* dev_meta, uint8_t* seg_is_pad,
                           int flags, void* stream);

/*
 * Dense-kernel eligibility of one ring chunk, on the GPU.
 *                           [cp_attention page, `_build_packed_ring_segments`
 *                            (the dense_local / dense_cross flags and pad_rows)
 *                            and `_chunk_dense_eligible`; the row predicates:
 *                            one document and no padding, or the real tokens
 *                            one document that forms a contiguous prefix with
 *                            padding only as a trailing suffix]
 *  kv_doc_ids: int32 [B, S] (1-based ids, 0 = padding); the query shard is
 *  [q_start, q_start + q_length) and the key chunk [k_start, k_start + k_length)
 *  of every row. Writes flags, a device int32[2], 1 = eligible:
 *   flags[0] (local role, causal): the chunk ends where the shard ends and
 *     contains it, and in every row the chunk's real tokens are one document
 *     forming a prefix (padding only as a suffix; an all-padding row counts).
 *     psf_attn_dense_fwd/bwd (causal) on the raw [B, H, N, D] shard and chunk,
 *     then psf_pad_fixup on the shard's ids, give the document-causal result.
 *   flags[1] (cross role, non-causal): the chunk lies before the shard, in
 *     every row [k_start, q_start) is one document d > 0 without padding, and
 *     the shard starts with d and holds no other document (padding only as a
 *     suffix). The non-causal dense kernels, then psf_pad_fixup, give the
 *     result of the psf_build_cross_segments segments.
 *  Errors: PSF_EINVAL when the shard or the chunk leaves the row.
 */
int psf_chunk_dense_flags(const int32_t* kv_doc_ids, int B, int S, int q_start, int q_length, int k_start,
                          int k_length, int32_t* flags, void* stream);

/*
 * Zero the padding queries of a document-causal result: rows whose query
 * document id is 0 get out = 0 and lse = -inf.
 *                           [fa4 page, `document_causal_fa4_attention`:
 *                            padding queries give zero output; cp_attention
 *                            page: rows that take no part get lse = -inf]
 *  q_doc_ids: int32 [B, Lq]; out / lse in `layout` with S = Lq.
 */
int psf_pad_fixup(void* out, float* lse, const int32_t* q_doc_ids, int layout, int B, int Lq, int Hq, int Dv,
                  void* stream);

/*
 * Merge two partial attention results computed over disjoint key sets.
 *                           [cp_attention page, "-inf-safe online-softmax merge"]
 *  l = logaddexp(l1, l2); o = o1 * exp(l1 - l) + o2 * exp(l2 - l), in fp32. A
 *  row with both inputs -inf gives o = 0, l = -inf (never NaN).
 *  o1, o2: dtype [T, H, D]; l1, l2: fp32 [H, T] (PSF_LAYOUT_THD only).
 *  Outputs: o_f32 (nullable) fp32 [T,H,D], o_bf16 (nullable) dtype [T,H,D],
 *  l fp32 [H,T]. Outputs may alias neither input.
 */
int psf_lse_merge(const void* o1, const float* l1, const void* o2, const float* l2, float* o_f32, void* o_bf16,
                  float* l, int T, int H, int D, int dtype, void* stream);

/*
 * Cross-chunk segments of a query shard against an earlier key chunk, on the
 * GPU (the one-device core of the ring decomposition).
 *                           [cp_attention page, `_build_packed_ring_segments`:
 *                            for each document present in both the query shard
 *                            and the KV chunk, its query tokens are paired with
 *                            its key tokens as one segment, cu_q[i] pairing
 *                            cu_k[i]; the chunk before the shard runs without a
 *                            causal mask]
 *  kv_doc_ids: int32 [B, S] document ids (1-based, 0 = padding, no document).
 *  The shard is [q_start, q_start + q_length) and the chunk
 *  [k_start, k_start + k_length) of every row, with the chunk before the shard
 *  (k_start + k_length <= q_start); the shard's queries and the chunk's keys are
 *  packed row-major as B * q_length and B * k_length rows. Since documents are
 *  contiguous runs, only the run holding position q_start can be shared. Each
 *  row gives three segments: (no queries x the chunk keys before the shared
 *  run), (the run's shard queries x its chunk keys), (the remaining shard
 *  queries x no keys); with nothing shared the middle one is empty.
 *  Outputs: cu_q, cu_k int32 [3 B + 1]; dev_meta int32[3] = {3 B, max_q, max_k}.
 *  Run the chunk with psf_attn_varlen_fwd/bwd, causal = 0: shard queries outside
 *  the shared run get out = 0, lse = -inf, dq = 0.
 *  Errors: PSF_EINVAL when the chunk does not lie before the shard.
 */
int psf_build_cross_segments(const int32_t* kv_doc_ids, int B, int S, int q_start, int q_length, int k_start,
                             int k_length, int32_t* cu_q, int32_t* cu_k, int32_t* dev_meta, void* stream);

/*
 * Merge one key chunk's result into a running result, in place, on the query
 * rows that took part in the chunk.
 *                           [cp_attention page, the in-place live-row merge of
 *                            a varlen chunk into the running accumulators at its
 *                            rows only, with the online-softmax merge]
 *  Live rows: the query rows of segments (cu_q, cu_k) that have at least one
 *  key. On those rows l = logaddexp(l_acc, l_new) and o = o_run exp(l_acc - l)
 *  + o_new exp(l_new - l) (both -inf gives o = 0, l = -inf); other rows are not
 *  touched. Running output: o_acc fp32 [T, H, D] (nullable) and/or o_run dtype
 *  [T, H, D] (nullable), read from o_acc when given, written to both; l_acc fp32
 *  [H, T] in place. o_new dtype [T, H, D], l_new fp32 [H, T]. No two of o_acc,
 *  o_run, o_new alias one another, nor l_acc and l_new.
 *  Segments: nseg (or dev_meta[0], capped at nseg, when dev_meta is given).
 */
int psf_lse_merge_live_rows(float* o_acc, void* o_run, float* l_acc, const void* o_new, const float* l_new,
                            const int32_t* cu_q, const int32_t* cu_k, const int32_t* dev_meta, int nseg, int T, int H,
                            int D, int dtype, void* stream);

/*
 * Add one key chunk's query gradient into the running one on the query rows
 * that took part in the chunk.
 *                           [cp_attention page, the in-place grad scatter-add
 *                            of a chunk's packed gradient into the full one]
 *  dst += src on the live rows of (cu_q, cu_k) (as in psf_lse_merge_live_rows),
 *  dtype [T, H, D] both, added in fp32 and rounded once; other rows untouched.
 *  dst and src do not alias.
 */
int psf_grad_add_live_rows(void* dst, const void* src, const int32_t* cu_q, const int32_t* cu_k,
                           const int32_t* dev_meta, int nseg, int T, int H, int D, int dtype, void* stream);

/*
 * Position rotation of queries and keys, forward and backward.
 *                           [no counterpart on the pages: an addition of this
 *                            library; it goes in front of the attention calls,
 *                            or of the cache's append]
 *
 *  Components [start, start + dim) of a head are dim / 2 pairs: (i, i + dim / 2)
 *  or, interleaved, (2 i, 2 i + 1), counted from start. Pair i of a row is turned
 *  by the angle a = position * inv_freq[i]:
 *    x0' = scale (x0 cos a - x1 sin a),  x1' = scale (x1 cos a + x0 sin a),
 *  in fp32, rounded once; the other components keep their values. The backward
 *  call turns by -a with the same scale, which is the transpose.
 *  inv_freq: fp32 [dim / 2] on the DEVICE, radians per position, below 2^62 in
 *  magnitude (a larger one, or one that is not finite, makes its pairs NaN). The
 *  angle is exact for any int32 position: it is reduced in 64-bit integers.
 *  axes: uint8 [dim / 2] on the HOST, the axis (0 to 7) that each pair takes its
 *  position from, or NULL (all axis 0); read during the call.
 *  dim is even, 2 to 512; scale is finite and > 0.
 */
typedef struct {
  const float* inv_freq;
  const uint8_t* axes;
  int dim, start, interleaved;
  float scale;
} psf_rotary;

/*
 *  q [T, Hq, D], k [T, Hkv, D] (dtype, PSF_LAYOUT_THD; or [B, H, S, D],
 *  PSF_LAYOUT_BHSD, with rows b * S + s) -> q_out, k_out of the same shape; dq and
 *  dk likewise. Hq or Hkv may be 0 (its pointers are not read). A result may be its
 *  input itself, with the same strides; otherwise it overlaps no input, and never the
 *  other tensor or its result (PSF_EINVAL where they begin at one address). D is a
 *  multiple of 8 up to 1024.
 *  Positions, in one of three ways:
 *    positions int32 [axes, rows] (axes 1 to 8; 1: every pair takes it whatever its axis);
 *    cu_seqlens int32 [nseg + 1], prefix sums over the rows: a row's place in its
 *      segment, for every axis. dev_meta (nullable): the count is dev_meta[0], and
 *      nseg the capacity, as for psf_attn_varlen_fwd. Rows past the last segment
 *      have position 0. Sums that fall, do not begin at 0 or pass the rows are a
 *      PSF_EDEVICE_ARGS status;
 *    neither: a row's place s in its batch row.
 *  A segment is all that these calls know of a document: where rows are a shard that
 *  begins inside one (psf_build_doc_segments with q_global_start > 0), the places of
 *  its cu_q begin at the shard's edge, not at the document's. psf_rotary_varlen_fwd
 *  and _bwd take such rows, and so do positions.
 *  strides: NULL, or 12 element strides (batch, head, row) of q, k, q_out, k_out.
 */
int psf_rotary_fwd(const void* q, const void* k, void* q_out, void* k_out, const psf_rotary* rotary,
                   const int32_t* positions, int axes, const int32_t* cu_seqlens, const int32_t* dev_meta, int nseg,
                   int layout, int B, int S, int Hq, int Hkv, int D, const int64_t* strides, int dtype, void* stream);
int psf_rotary_bwd(const void* dq, const void* dk, void* dq_out, void* dk_out, const psf_rotary* rotary,
                   const int32_t* positions, int axes, const int32_t* cu_seqlens, const int32_t* dev_meta, int nseg,
                   int layout, int B, int S, int Hq, int Hkv, int D, const int64_t* strides, int dtype, void* stream);

/*
 * psf_rotary_fwd and _bwd with query rows placed as psf_attn_varlen_fwd aligns them
 * to their keys: row i of the m rows [cu_q[s], cu_q[s + 1]) of segment s, which has
 * n = cu_k[s + 1] - cu_k[s] keys, has position i + n - m (negative in a padding run
 * without keys). cu_q and cu_k int32 [nseg + 1] as psf_build_doc_segments writes
 * them, for any shard; dev_meta (nullable) as above. cu_k that falls or does not
 * begin at 0 is a PSF_EDEVICE_ARGS status, too. The keys themselves: psf_rotary_fwd
 * with cu_k as their cu_seqlens, which places every key that a row of the shard sees.
 * (A document that goes on past the shard's end has a second segment there, without
 * queries, whose places begin anew.)
 */
int psf_rotary_varlen_fwd(const void* q, const void* k, void* q_out, void* k_out, const psf_rotary* rotary,
                          const int32_t* cu_q, const int32_t* cu_k, const int32_t* dev_meta, int nseg, int layout, int B,
                          int S, int Hq, int Hkv, int D, const int64_t* strides, int dtype, void* stream);
int psf_rotary_varlen_bwd(const void* dq, const void* dk, void* dq_out, void* dk_out, const psf_rotary* rotary,
                          const int32_t* cu_q, const int32_t* cu_k, const int32_t* dev_meta, int nseg, int layout, int B,
                          int S, int Hq, int Hkv, int D, const int64_t* strides, int dtype, void* stream);

/*
 * 8-bit paged key/value cache, for serving: append, attention of a few query
 * rows per sequence, eviction by accumulated attention weight, gather.
 *                           [no counterpart on the pages: an addition of this
 *                            library; the attention is the varlen forward's
 *                            (scale, softcap, causal alignment, left window, lse)]
 *
 *  A cache is a pool of pages. A page holds page_size tokens (16, 32, 64 or 128)
 *  of every KV head as e4m3 codes, with one fp32 scale per (page, head) for K
 *  and one for V: a code c stands for the value c * scale.
 *    k [num_pages, Hkv, page_size, Dqk], v [num_pages, Hkv, page_size, Dv] e4m3,
 *    k_scale, v_scale [num_pages, Hkv] fp32 (finite, >= 0), contiguous,
 *    weight [num_pages, Hkv, page_size] fp32, contiguous, or NULL: the attention
 *    weight each token has received so far, for eviction.
 *  k_strides / v_strides: element strides (page, head, row), all zero for the
 *  contiguous ones; else positive multiples of 16 below 2^38 (a dimension of
 *  extent 1 is ignored), and no overlap. The last dim is contiguous; k, v and
 *  weight are 16-byte aligned. Head dims as for the attention calls. Append and
 *  eviction change K and V at the same time and need them in memory of their own
 *  (PSF_EINVAL where k is v or the scales overlap); the others only read them.
 *
 *  Sequences: page_table int32 [B, max_pages] (contiguous) lists the pages of
 *  each sequence in order, seq_lens int32 [B] its tokens: token j of sequence b
 *  is row j % page_size of page page_table[b][j / page_size]. Entries past
 *  ceil(seq_lens[b] / page_size) are not read. max_pages * page_size is at most
 *  2^31 - 2^16. Several sequences may name the
 *  same page (a shared prefix) as long as no call writes to it. All of it is
 *  read on the device: nothing synchronises, and the calls can be captured.
 *  A length outside [0, max_pages * page_size], prefix sums that do not begin at 0
 *  or whose rows lie outside the packed tensor, or a page outside [0, num_pages)
 *  is a PSF_EDEVICE_ARGS device status; nothing outside the tensors is touched, a
 *  page that does not exist is not written, and the results of the other
 *  sequences stand (but see the append for its prefix sums).
 */
typedef struct {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  float* weight;
  int num_pages, page_size, Hkv, Dqk, Dv;
  int64_t k_strides[3], v_strides[3];
} psf_kv_cache;

/*
 * Quantise new rows into the cache.
 *  k [T, Hkv, Dqk], v [T, Hkv, Dv] (dtype): the new tokens of all sequences,
 *  packed; sequence b's are rows [cu_new[b], cu_new[b + 1]) (int32 [B + 1]), or,
 *  with cu_new NULL, T / B rows each (B must divide T). seq_lens counts them
 *  already: they go to positions seq_lens[b] - n_b .. seq_lens[b] - 1.
 *  Scale: s(a) is the smallest power of two >= 2^-126 with a <= 448 s. A page
 *  whose first row is new gets s(largest finite magnitude of its new rows); a
 *  page that holds older tokens of the sequence gets the larger of its scale and
 *  that, and where it grows the older codes c become RNE_e4m3(c * (old / new)),
 *  exact down to the format's subnormals. New codes are RNE_e4m3(x / scale); a
 *  value that is not finite becomes NaN. The weights of new tokens become 0.
 *  Rows of T past cu_new[B] are not read; rows of a page past the new ones keep
 *  their contents. A page that is written belongs to one sequence. A sequence
 *  with more new rows than tokens takes none (a PSF_EDEVICE_ARGS status): idle
 *  entries of a batch have no rows in cu_new.
 *  Pages are looked up by prefix sums, so where one falls below the entry in front
 *  of it or passes T, new rows of any sequence may be left out.
 *  strides: NULL, or 6 element strides (batch, head, row) of k, v (batch ignored).
 */
int psf_kv_cache_append(const psf_kv_cache* cache, const void* k, const void* v, const int64_t* strides, int dtype,
                        const int32_t* cu_new, const int32_t* page_table, const int32_t* seq_lens, int B,
                        int max_pages, int T, void* stream);

/*
 * The append of new rows whose keys are turned on the way (see psf_rotary).
 *  As psf_kv_cache_append, with the keys' turned values, kept in fp32 until they
 *  become codes, in place of k's. q [T, Hq, Dqk] (Hq 0: none), the queries of the
 *  same tokens, are turned into q_out in the same call (q_out may be q itself;
 *  otherwise it overlaps no input: PSF_EINVAL where it begins at k or v).
 *  positions int32 [axes, T] as for psf_rotary_fwd, or NULL with axes 0: a token's
 *  place in its sequence, 0 for rows of no sequence. After an eviction places
 *  count kept tokens, so a cache that is evicted from wants positions.
 *  strides: NULL, or 12 element strides (batch, head, row) of k, v, q, q_out (batch ignored).
 */
int psf_kv_cache_append_rotary(const psf_kv_cache* cache, const void* k, const void* v, const void* q, void* q_out,
                               const psf_rotary* rotary, const int32_t* positions, int axes, const int64_t* strides,
                               int dtype, const int32_t* cu_new, const int32_t* page_table, const int32_t* seq_lens,
                               int B, int max_pages, int T, int Hq, void* stream);

/*
 * Attention of packed query rows over the cache.
 *  q [T, Hq, Dqk], out [T, Hq, Dv] (dtype), lse [Hq, T] fp32. Sequence b's query
 *  rows are [cu_q[b], cu_q[b + 1]), or T / B each with cu_q NULL; max_q: the most
 *  rows of a sequence (more is a PSF_EDEVICE_ARGS status). They are the last
 *  tokens of the sequence: row i of m sits at position seq_lens[b] - m + i, the
 *  bottom-right alignment of the causal mask and the window. scale, causal,
 *  window_left, softcap, GQA and rows without keys as for psf_attn_varlen_fwd;
 *  rows past cu_q[B] get out = 0 and lse = -inf.
 *  One query row per sequence is the decode step; a few are drafted tokens or the
 *  tail of a prompt. Any number is computed, a tile of rows at a time; for long
 *  prompt chunks psf_attn_cache_prompt_fwd is faster, and at head dim 512
 *  psf_kv_cache_gather with psf_attn_varlen_fwd.
 *  Codes that are NaN make a row NaN only where it sees them.
 *  flags: 0, or PSF_CACHE_ACCUMULATE: weight[page, hkv, row] += the sum over the
 *  sequence's query rows and the Hq / Hkv heads of hkv of exp(logit - lse), for
 *  every token seen. With a page in several sequences the order of the additions
 *  is not fixed. Other bits: PSF_EINVAL.
 *  strides: NULL, or 6 element strides (batch, head, row) of q, out (batch ignored).
 *  workspace: psf_attn_cache_workspace_size(...) bytes, 16-byte aligned; nothing in it
 *  has to be kept or cleared between calls. (With PSF_CACHE_ACCUMULATE it holds the
 *  scores, 4 B * Hq * max_q * max_pages * page_size bytes more; SIZE_MAX where no memory holds them.)
 */
#define PSF_CACHE_ACCUMULATE 1
size_t psf_attn_cache_workspace_size(int B, int max_pages, int page_size, int Hq, int Hkv, int Dqk, int Dv,
                                     int max_q, int flags);
int psf_attn_cache_fwd(const void* q, const psf_kv_cache* cache, void* out, float* lse, const int32_t* cu_q,
                       const int32_t* page_table, const int32_t* seq_lens, int B, int max_pages, int T, int max_q,
                       int Hq, const int64_t* strides, int dtype, float scale, int causal, int32_t window_left,
                       float softcap, int flags, void* workspace, size_t ws_bytes, void* stream);

/*
 * Attention of prompt chunks over the cache: what psf_attn_cache_fwd computes,
 * on the tensor cores' 256-row tiles, for sequences with many query rows.
 *  Arguments, results, masks and statuses as there, without flags (no weights are
 *  accumulated: before an eviction, tokens of a chunk have only what later calls of
 *  psf_attn_cache_fwd add). A KV head's query heads share its tiles, so a batch may mix
 *  chunks, tails and single tokens. The kernel of psf_attn_cache_fwd runs where it
 *  is the faster one: for at most 32 rows per KV head (max_q * Hq / Hkv), and where
 *  little is to be done (B * Hkv * rows / 16 * max_pages * page_size up to 4 * 10^5:
 *  by the table's width, as the lengths are on the device). It runs at head dim 512,
 *  too, which the tiles do not do.
 *  Faster through psf_kv_cache_gather and psf_attn_varlen_fwd, where there is memory
 *  for the 16-bit copies: long chunks at head dim 512 (two of 2048 rows over 32 Ki
 *  keys, 8 / 2 heads: 3.7 ms for 13.9 here), hundreds of short sequences (2000 whole
 *  prompts of 10 to 100 tokens: 0.63 ms for 1.21) and whole prompts at 192/128 (two
 *  of 8001 with a window: 0.50 for 0.55). Decode steps are faster in a call of their
 *  own than beside a chunk (63 with a chunk of 512 over 8 Ki keys: 292 us for 467).
 *  P is rounded to fp16 whatever the dtype; queries are scaled by a power of two
 *  per row into fp16's range. The same call gives the same bits; under a softcap a
 *  row's last bits may depend on the rows that share its tile.
 *  workspace: psf_attn_cache_prompt_workspace_size(...) bytes, 16-byte aligned (42 MB
 *  at head dim 128, whatever the batch); nothing in it has to be kept or cleared between calls.
 */
size_t psf_attn_cache_prompt_workspace_size(int B, int max_pages, int page_size, int Hq, int Hkv, int Dqk, int Dv,
                                            int max_q);
int psf_attn_cache_prompt_fwd(const void* q, const psf_kv_cache* cache, void* out, float* lse, const int32_t* cu_q,
                              const int32_t* page_table, const int32_t* seq_lens, int B, int max_pages, int T, int max_q,
                              int Hq, const int64_t* strides, int dtype, float scale, int causal, int32_t window_left,
                              float softcap, void* workspace, size_t ws_bytes, void* stream);

/*
 * Evict down to `budget` tokens per sequence and KV head, in place.
 *  A sequence longer than budget keeps, for each KV head on its own, its last
 *  `recent` tokens and the budget - recent others of largest weight (of equal
 *  weights the earliest; NaN counts as the largest, -0 as 0), in their order, moved to
 *  positions 0 .. budget - 1; weights move along. new_lens[b] = min(seq_lens[b],
 *  budget); other sequences are not touched. A new block's scale is the largest
 *  old scale of its tokens, codes become RNE_e4m3(c * r), r = old / new in fp32 (exact
 *  for powers of two, the scales that the append chooses). Rows past the
 *  kept ones keep their contents; pages past ceil(budget / page_size) are free.
 *  After an eviction positions count kept tokens (so do windows).
 *  A sequence with a page that does not exist is left as it is, its new length
 *  its old one. Needs cache->weight, 1 <= budget, 0 <= recent <= budget. new_lens
 *  must not overlap seq_lens. A page belongs to one sequence.
 *  workspace: psf_kv_cache_evict_workspace_size(...) bytes, 16-byte aligned.
 */
size_t psf_kv_cache_evict_workspace_size(int B, int max_pages, int page_size, int Hkv, int budget);
int psf_kv_cache_evict(const psf_kv_cache* cache, const int32_t* page_table, const int32_t* seq_lens,
                       int32_t* new_lens, int B, int max_pages, int budget, int recent, void* workspace,
                       size_t ws_bytes, void* stream);

/*
 * The cached rows of all sequences as packed 16-bit tensors.
 *  k [total_k, Hkv, Dqk], v [total_k, Hkv, Dv] (dtype, contiguous): row
 *  cu_k[b] + j is token j of sequence b, code * scale in fp32 rounded to the type
 *  (with scales written by the append, exact in bf16). cu_k int32 [B + 1]: prefix sums of
 *  seq_lens. With q, cu_k and these the varlen forward attends a long prompt
 *  chunk over its cached prefix. total_k bounds the sum of the lengths (more is a
 *  PSF_EDEVICE_ARGS status, and the rows past it are dropped); rows past cu_k[B]
 *  are not written.
 */
int psf_kv_cache_gather(const psf_kv_cache* cache, const int32_t* page_table, const int32_t* seq_lens, int B,
                        int max_pages, void* k, void* v, int32_t* cu_k, int total_k, int dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PSF_H_ */
