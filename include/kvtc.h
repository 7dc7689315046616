/*
 * kvtc.h -- C ABI of the GB300 (sm_103a) KV-cache transform codec.
 *
 * The method is KV-cache transform coding ("KV Cache Transform Coding for
 * Compact Storage in LLM Inference", technical summary section 2):
 *   compress    (2B)  c = V^T (x - mu), keep the principal components whose
 *                     group the DP allocation gave a nonzero width, quantise
 *                     each 16-component group with an fp16 shift and scale
 *                     of its own (microscaling, 2A), pack the codes;
 *   decompress  (2C)  unpack, dequantise, x_hat = V c_hat + mu, bf16;
 *   sinks/window (2A) the first s and the last w tokens are stored raw.
 * The DEFLATE stage the page runs after packing (2B) is not part of this
 * library; an optional lossless field-packing stage of its own is
 * (kvtc_fields_pack / kvtc_fields_unpack).
 *
 * Conventions for every entry point:
 *   - All device pointers are caller-owned CUDA device memory on the device
 *     the calibration was loaded on.  The library allocates device memory
 *     only in kvtc_calib_load (and frees it in kvtc_calib_free); the codec
 *     calls allocate nothing.
 *   - Work is enqueued on the caller's stream (a cudaStream_t passed as
 *     void*; NULL = the legacy default stream).  KVTC_OK means "validated
 *     and enqueued", not "finished".
 *   - Arguments are validated on the host before any launch; on error
 *     nothing is enqueued and a negative status is returned.
 *   - Faults detected by the kernels (fp16 field overflow, a block id out
 *     of range, a bounded wait that ran out) never trap: the kernel skips
 *     the affected write and ORs a flag into a sticky per-calibration status
 *     word, read and cleared with kvtc_device_status.
 *   - Pointers that the kernels reach with 16-byte vector or bulk copies
 *     must be 16-byte aligned, and row strides (ld) multiples of 8 elements.
 *   - The calls are thread-safe on the host, and a launch's parameters
 *     travel with the launch (nothing is staged in library-owned memory).
 *     A loaded calibration is read-only on the device, so codec calls that
 *     use it may run at the same time on several streams; their kernel
 *     flags all land in its one status word.  The one exception is
 *     kvtc_calib_mean_static (below).
 *
 * Formats (all little-endian):
 *
 *   Token record (R = 16 * ceil(budget_bits / 128) bytes): for each active
 *   group g in ascending order a u16 fp16 shift then a u16 fp16 scale; then
 *   for each active group in ascending order its b_g bit-planes, one u16
 *   each, bit i of plane j = bit j of the code of the group's i-th
 *   component; zero padding to R.  Code q of coefficient c:
 *     shift = fp16 round-down of the group minimum,
 *     scale = fp16 round-up of (max - shift) / (2^b - 1),
 *     q = clamp(floor((c - shift) / scale + 1/2), 0, 2^b - 1)  (0 if scale 0),
 *     c_hat = shift + q * scale.
 *
 *   Stream of one (request, layer, K|V) with T tokens, s' = min(s, T),
 *   w' = min(w, T - s'), T_c = T - s' - w':  s' sink rows (bf16 [s'][D]),
 *   w' window rows (bf16 [w'][D]), T_c records in token order; the stream
 *   is padded to a multiple of 256 bytes.  Several streams are concatenated
 *   in (layer, K, V) order.
 *
 *   Calibration blob, version 1: "KVTC", u32 version, n_streams, group (16),
 *   bmax (8), sink, window, budget_bits; per stream u32 layer, kv (0 = K,
 *   1 = V), D, k, u8 widths[D/16] zero-padded to a multiple of 8 bytes, f64
 *   mu[D], f64 V_kept[k][D] (row a = a-th kept principal vector, ascending
 *   component order), f64 eigenvalues[D]; trailer u32 CRC-32 (IEEE 802.3) of
 *   all preceding bytes, u32 0.
 */
#ifndef KVTC_H
#define KVTC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum kvtc_status {
  KVTC_OK = 0,
  KVTC_EINVAL = -1,   /* null/invalid argument, layer or kv not in blob */
  KVTC_EFORMAT = -2,  /* blob magic/version/checksum/structure */
  KVTC_ESIZE = -3,    /* buffer too small, sizes inconsistent */
  KVTC_ENOMEM = -4,   /* device allocation in kvtc_calib_load failed */
  KVTC_ECUDA = -5,    /* a CUDA runtime/driver call failed */
  KVTC_ERANGE = -6,   /* device flag: fp16 field overflow in compress */
  KVTC_EDEVICE = -7,  /* device flag: bounded wait ran out / bad block id */
  KVTC_EALIGN = -8,   /* pointer or stride misaligned */
  KVTC_ENOTSUP = -9   /* shape outside what the kernels support */
};

/* Sticky device flags reported by kvtc_device_status (bit mask). */
#define KVTC_FLAG_RANGE 1u     /* a shift/scale left the fp16 range */
#define KVTC_FLAG_TIMEOUT 2u   /* a bounded mbarrier wait ran out */
#define KVTC_FLAG_BLOCK 4u     /* block-table id outside [0, num_blocks) */
#define KVTC_FLAG_FORMAT 8u    /* packed stream inconsistent (field packing) */
#define KVTC_FLAG_SPACE 16u    /* free list, block table or slot map too short */

/* Element type of a paged pool read by kvtc_paged_attend. */
enum kvtc_dtype {
  KVTC_DTYPE_BF16 = 0,
  KVTC_DTYPE_FP16 = 1
};

typedef struct kvtc_calib kvtc_calib;

/*
 * kvtc_calib_load -- parse a calibration blob and build the device operands.
 * Reading of technical summary 2A: mu, the basis V and the per-group widths
 * come from a one-time calibration and are shared by every request.
 *   blob, blob_bytes : host memory, read only during the call.
 *   cuda_device      : device ordinal that will run the codec.
 *   out              : receives an opaque handle (owned by the caller, free
 *                      with kvtc_calib_free).
 * Derived on load: bf16 V_kept (projection), fp16 V_kept (reconstruction),
 * fp32 mu and fp32 m = bf16(V_kept) mu, group layout tables, TMA
 * descriptors.  Requirements: D % 64 == 0, D <= 8192, 16 <= k <= 496 (the
 * reconstruction holds k plus one mean step of 16 fp16 columns in 256
 * tensor-memory columns) and record bytes <= 256; otherwise ENOTSUP.  Up
 * to k = 240 both kernels double-buffer their tensor-memory operands;
 * above, a launch that holds such a stream single-buffers them (the
 * projection above k = 256, the reconstruction's A operand above k = 240).
 * The projection's shared-memory ring holds two or more stages while
 * 2 (32768 + 128 k) + 264 R + 1344 <= 232448 bytes (k <= 382 at R = 256),
 * one stage beyond.
 * Errors: EINVAL, EFORMAT, ENOMEM, ECUDA, ENOTSUP.
 */
int kvtc_calib_load(const void* blob, size_t blob_bytes, int cuda_device,
                    kvtc_calib** out);
void kvtc_calib_free(kvtc_calib* calib);

/* Shape of stream (layer, kv): D, kept components k, sink s, window w,
 * record bytes R.  Any output pointer may be NULL.  EINVAL if absent. */
int kvtc_calib_query(const kvtc_calib* calib, int layer, int kv, int* D,
                     int* k, int* s, int* w, int* record_bytes);

/* Bytes of one stream of T tokens (multiple of 256); < 0 on error. */
int64_t kvtc_stream_bytes(const kvtc_calib* calib, int layer, int kv,
                          int64_t T);

/*
 * kvtc_compress -- technical summary 2B (and 2A for sinks/window).
 *   layer0, nlayers : layers [layer0, layer0 + nlayers).
 *   kv_mask         : 1 = K, 2 = V, 3 = both.
 *   src             : HOST array of 2*nlayers device pointers, entry
 *                     2*(l - layer0) + kv = bf16 [T][ld] rows of that stream
 *                     (entries of kinds not in kv_mask are ignored).
 *   ld              : row stride of src in elements (>= D, % 8 == 0).
 *   T               : tokens (>= 0).
 *   dst, dst_bytes  : device output; streams concatenated in (layer, K, V)
 *                     order, each kvtc_stream_bytes long.
 * Errors: EINVAL, ESIZE, EALIGN, ECUDA, ENOTSUP.
 */
int kvtc_compress(const kvtc_calib* calib, int layer0, int nlayers,
                  int kv_mask, const void* const* src, int64_t ld, int64_t T,
                  void* dst, int64_t dst_bytes, void* cuda_stream);

/*
 * kvtc_decompress -- technical summary 2C.
 *   src, src_bytes  : input written by kvtc_compress (same layers, kv_mask
 *                     and T), in device memory or in pinned host memory
 *                     (cudaHostAlloc / cudaHostRegister).  Pinned host
 *                     memory is read by the kernels themselves over the
 *                     host link (on GB300, NVLink-C2C), with no staging
 *                     copy.  Pageable host memory: EINVAL.
 *   dst             : HOST array of 2*nlayers device pointers (as src of
 *                     kvtc_compress), each bf16 [T][ld].
 *   layer_events    : NULL, or a HOST array of nlayers cudaEvent_t (as
 *                     void*).  When given, layers are restored one launch
 *                     per layer in order and event l is recorded once layer
 *                     layer0 + l is complete, so a consumer can start on
 *                     early layers (layer-wise decompression, 2C).
 * Errors: EINVAL, ESIZE, EALIGN, ECUDA, ENOTSUP.
 */
int kvtc_decompress(const kvtc_calib* calib, int layer0, int nlayers,
                    int kv_mask, const void* src, int64_t src_bytes,
                    int64_t T, void* const* dst, int64_t ld,
                    void* cuda_stream, void* const* layer_events);

/*
 * kvtc_decompress_paged -- restore R requests into a paged KV pool (the
 * block-paged prefix cache of technical summary section 1).
 *   src          : HOST array [R] of pointers; src[r] holds request r's
 *                  streams as kvtc_compress wrote them, in device memory or
 *                  pinned host memory (as for kvtc_decompress).
 *   T            : HOST array [R] of token counts.
 *   block_table  : DEVICE int32 [R][max_blocks]; token t of request r goes
 *                  to block block_table[r*max_blocks + t/block_size], row
 *                  t % block_size.  Ids outside [0, num_blocks) are skipped
 *                  and flag KVTC_FLAG_BLOCK.
 *   block_size   : tokens per block; 16 (other sizes return ENOTSUP).
 *   max_blocks   : columns of block_table; every request needs
 *                  ceil(T[r] / block_size) of them (ESIZE otherwise).
 *   cache        : HOST array of 2*nlayers device pointers, each bf16
 *                  [num_blocks][block_size][D] (entries of kinds not in
 *                  kv_mask ignored).
 * All selected streams must share one D.  R <= 4096 (split larger sets).
 * Errors: EINVAL, ESIZE, EALIGN, ECUDA, ENOTSUP.
 */
int kvtc_decompress_paged(const kvtc_calib* calib, int layer0, int nlayers,
                          int kv_mask, const void* const* src,
                          const int64_t* T, int R, const int32_t* block_table,
                          int max_blocks, int block_size, void* const* cache,
                          int64_t num_blocks, void* cuda_stream);

/*
 * Field packing -- a lossless stage after bit-packing.  The page runs DEFLATE
 * there (technical summary 2B); this library runs a format of its own that
 * targets the one redundant part of a record, the high byte of each fp16
 * field.  Per stream and field slot (slot 2a = shift of active group a,
 * 2a + 1 = its scale), v = high byte h >> 2 (sign and exponent) spans
 * [vmin, vmin + 2^dbits) over the stream's records (dbits <= 6), so h is
 * stored as h - 4 vmin in dbits + 2 bits; the other bits are kept, and the
 * record's zero padding is dropped.
 *
 *   Packed stream (little-endian): header "KVFP", u32 T_c, u16 Rp (packed
 *   record bytes), u16 nslot (= 2 G_a), u32 0; slot table nslot x (u8 vmin,
 *   u8 dbits) zero-padded so that header and table fill 128 bytes (a
 *   multiple of 128 above 56 slots); the s' + w' raw rows as in the codec
 *   stream; T_c packed records of Rp bytes; zeros to a 256-byte multiple.
 *   Packed record: the low bytes of the 2 G_a fields in slot order; the
 *   codes, per slot h - 4 vmin in dbits + 2 bits, least significant bit
 *   first, in 2 ceil(bits / 16) bytes; the bit-planes of the codec record
 *   unchanged; zeros to a multiple of 4 bytes.  Rp <= R, so a packed
 *   stream is never longer than the codec stream plus its 128-byte prefix.
 *   The records of a stream start on a 128-byte line and 32 of them fill
 *   whole lines, which the restore from packed input reads line by line.
 *   Streams are concatenated in (layer, K, V) order.
 */

/* Field packing holds one field slot per lane of a warp: every selected
 * stream must keep at most 15 groups (k <= 240), else the three calls below
 * return ENOTSUP. */

/* Upper bound on the packed bytes of the selected streams at T tokens
 * (< 0 on error). */
int64_t kvtc_fields_bound(const kvtc_calib* calib, int layer0, int nlayers,
                          int kv_mask, int64_t T);

/* Device workspace bytes kvtc_fields_pack needs (< 0 on error). */
int64_t kvtc_fields_workspace_bytes(const kvtc_calib* calib, int layer0,
                                    int nlayers, int kv_mask);

/*
 * kvtc_fields_pack -- pack codec streams.
 *   src, src_bytes   : device codec streams as kvtc_compress wrote them
 *                      (same layers, kv_mask and T).
 *   dst, dst_capacity: device output, at least kvtc_fields_bound bytes; the
 *                      packed streams are written back to back.
 *   offsets          : device int64 [n + 1] (n = selected streams), written:
 *                      packed stream i occupies [offsets[i], offsets[i+1])
 *                      of dst; offsets[n] is the packed size.
 *   workspace        : device scratch of kvtc_fields_workspace_bytes bytes,
 *                      used only while the call's work runs on cuda_stream.
 * Three kernel launches per 256 streams (a min/max pass, a layout pass that
 * writes headers, tables and offsets, and the pack pass); no host
 * synchronisation.  src, dst and workspace 16-byte aligned, offsets 8.
 * Errors: EINVAL, ESIZE, EALIGN, ENOMEM, ECUDA.
 */
int kvtc_fields_pack(const kvtc_calib* calib, int layer0, int nlayers,
                     int kv_mask, const void* src, int64_t src_bytes,
                     int64_t T, void* dst, int64_t dst_capacity,
                     int64_t* offsets, void* workspace,
                     int64_t workspace_bytes, void* cuda_stream);

/*
 * kvtc_fields_unpack -- restore the codec streams that kvtc_fields_pack
 * packed, byte for byte.
 *   src, src_bytes : device packed streams.
 *   offsets        : device int64 [n + 1] as kvtc_fields_pack wrote them.
 *   dst, dst_bytes : device output, the codec streams (kvtc_stream_bytes
 *                    each, concatenated as kvtc_compress writes them).
 * Each stream's header and table are checked against its calibration, T
 * and offsets on the GPU; a stream that does not match is skipped and flags
 * KVTC_FLAG_FORMAT.  One kernel launch per 256 streams.
 * Errors: EINVAL, ESIZE, EALIGN, ENOMEM, ECUDA.
 */
int kvtc_fields_unpack(const kvtc_calib* calib, int layer0, int nlayers,
                       int kv_mask, const void* src, int64_t src_bytes,
                       const int64_t* offsets, int64_t T, void* dst,
                       int64_t dst_bytes, void* cuda_stream);

/*
 * kvtc_decompress_packed -- the restore of kvtc_decompress (the mapping of
 * technical summary 2A inverted: dequantise, project back with V_kept^T, add
 * mu) read straight from the packed streams that kvtc_fields_pack wrote: the
 * restore kernel unpacks each record's fields as it loads it, so the packed
 * bytes are the only compressed bytes read and no codec stream is written.
 * The output is bit-identical to kvtc_fields_unpack followed by
 * kvtc_decompress.
 *   src, src_bytes : the packed streams, in device memory or pinned host
 *                    memory (read by the kernels over the host link, zero
 *                    copy); pageable host memory is refused (EINVAL).
 *   offsets        : int64 [n + 1] as kvtc_fields_pack wrote them (n =
 *                    selected streams), device or pinned host memory.
 *   T, dst, ld, cuda_stream, layer_events : as for kvtc_decompress.
 * Each stream's header, slot table and length are checked against its
 * calibration, T, the offsets and src_bytes on the GPU before anything they
 * frame is read; a stream that does not match restores its coded tokens as
 * from all-zero records and flags KVTC_FLAG_FORMAT.  Its raw rows are copied
 * whenever its extent frames them (both offsets on the 16-byte grid, inside
 * src_bytes), and, in a call with no coded token, only when its magic and
 * T_c check out too; an out-of-frame stream flags KVTC_FLAG_FORMAT.
 * Kernel launches as for kvtc_decompress (the raw rows of a call with no
 * coded token take one copy launch per 96 streams).  Streams must keep at
 * most 15 groups, else ENOTSUP.  src 16-byte aligned, offsets 8.
 * Errors: EINVAL, ESIZE, EALIGN, ENOTSUP, ENOMEM, ECUDA.
 */
int kvtc_decompress_packed(const kvtc_calib* calib, int layer0, int nlayers,
                           int kv_mask, const void* src, int64_t src_bytes,
                           const int64_t* offsets, int64_t T,
                           void* const* dst, int64_t ld, void* cuda_stream,
                           void* const* layer_events);

/*
 * Paged serving -- the calls around kvtc_decompress_paged in one serving
 * step: blocks and slots for the requests' tokens, rows of new tokens
 * written through the slots, and attention of one new token per request
 * over the pool.  They need no calibration: each takes the device ordinal
 * that owns its pointers (whatever device is current), allocates nothing,
 * keeps nothing between calls and never synchronises, so a call can be
 * captured into a CUDA graph and replayed with other lengths, ids and rows
 * in the same buffers.  Their kernels report faults into `flags`, a DEVICE
 * uint32 word of the caller's into which KVTC_FLAG_* bits are ORed (it is
 * never cleared here; NULL: faults are not reported).  Blocks hold 16
 * tokens (block_size 16, other sizes ENOTSUP), R <= 4096.
 */

/* Device workspace bytes kvtc_paged_assign needs (< 0 on error). */
int64_t kvtc_paged_assign_workspace_bytes(int R);

/*
 * kvtc_paged_assign -- give R requests the blocks that their tokens need,
 * in request order, and list the slots of the new tokens.
 *   held, lens   : DEVICE int32 [R]: tokens of request r that have blocks,
 *                  and tokens that it is to have; its new tokens are
 *                  held[r] .. lens[r] - 1 (none when lens[r] <= held[r],
 *                  negative values count as 0).
 *   free_blocks  : DEVICE int32 [n_free]: block ids, given out from the
 *                  front.  May be NULL when n_free is 0.
 *   head         : DEVICE int64 [1]: how many of them have been given out.
 *   block_table  : DEVICE int32 [R][max_blocks], as kvtc_decompress_paged
 *                  reads it: columns ceil(held[r] / 16) ..
 *                  ceil(lens[r] / 16) - 1 of a served request are written,
 *                  all others are left as they are.
 *   slots        : DEVICE int64 [slot_capacity], written whole: new token j
 *                  of request r at slots[cu[r] + j] is row
 *                  id * 16 + t % 16 of a pool seen as [num_blocks * 16][D]
 *                  (t = held[r] + j, id = block_table[r][t / 16]); -1 for a
 *                  token without a place (request not served, or a
 *                  negative id in the table) and behind the last token.
 *                  Tokens past slot_capacity get blocks but no entry.  May
 *                  be NULL when slot_capacity is 0.
 *   cu           : DEVICE int64 [R + 1], written: cu[r] = new tokens of the
 *                  requests before r, served or not; cu[R] = all of them.
 *   held_out     : DEVICE int32 [R], written: max(held[r], lens[r]) of a
 *                  served request, held[r] of another.  May be held itself.
 *   head_out     : DEVICE int64 [1], written: head plus the blocks given
 *                  out.  May be head itself.
 * A request is served unless lens[r] > 16 * max_blocks (it then takes no
 * block), or it needs blocks and the requests up to and including it need
 * more than free_blocks still holds.  A request with new tokens that is not
 * served, new tokens past slot_capacity, and head outside [0, n_free] (then
 * no block is given out) flag KVTC_FLAG_SPACE.  Other than as said, no
 * output may overlap an input or another output.
 * workspace: device scratch of kvtc_paged_assign_workspace_bytes bytes, used
 * only while the call's work runs on cuda_stream, 16-byte aligned; slots, cu,
 * head and head_out are 8-byte aligned, the int32 arrays 4.  One kernel
 * launch for up to 1024 requests, unless slot_capacity is above 16 R (or
 * 8192) or below R / 2 and held_out is held or head_out is head; else two.
 * Errors: EINVAL, ESIZE, EALIGN, ENOTSUP, ECUDA.
 */
int kvtc_paged_assign(int cuda_device, int R, const int32_t* held,
                      const int32_t* lens, const int32_t* free_blocks,
                      int64_t n_free, const int64_t* head,
                      int32_t* block_table, int max_blocks, int block_size,
                      int64_t* slots, int64_t slot_capacity, int64_t* cu,
                      int32_t* held_out, int64_t* head_out, void* workspace,
                      int64_t workspace_bytes, uint32_t* flags,
                      void* cuda_stream);

/*
 * kvtc_paged_append -- write rows of new tokens into paged pools: row i of
 * stream j goes to row slots[i] of cache[j] seen as [num_blocks * 16][D].
 *   nstreams : streams (K and V of a layer, or of several layers); >= 0.
 *   src      : HOST array [nstreams] of device pointers, stream j's rows:
 *              16-bit elements (bf16 or fp16, copied bit for bit) [N][ld].
 *   ld       : row stride of every src in elements (>= D, % 8 == 0), so the
 *              streams may be column slices of one projection's rows.
 *   slots    : DEVICE int64 [N], as kvtc_paged_assign lists them.  Negative:
 *              the row is skipped.  At or past num_blocks * 16: skipped, and
 *              KVTC_FLAG_BLOCK is set.  The others must be distinct: of two
 *              rows with one slot, either may supply each 16 bytes of it.
 *   cache    : HOST array [nstreams] of device pointers, each 16-bit
 *              [num_blocks][16][D]; rows that no slot names are untouched.
 * D % 8 == 0, 8 <= D <= 8192.  src and cache 16-byte aligned, slots 8.  No
 * cache may overlap another, a src or slots.  One kernel launch per 64
 * streams.
 * Errors: EINVAL, ESIZE, EALIGN, ENOTSUP, ECUDA.
 */
int kvtc_paged_append(int cuda_device, int nstreams, const void* const* src,
                      int64_t ld, int64_t N, const int64_t* slots, int D,
                      int block_size, void* const* cache, int64_t num_blocks,
                      uint32_t* flags, void* cuda_stream);

/* Device workspace bytes kvtc_paged_attend needs (< 0 on error). */
int64_t kvtc_paged_attend_workspace_bytes(int cuda_device, int R, int heads,
                                          int kv_heads, int head_dim);

/*
 * kvtc_paged_attend -- attention of one new token of each of R requests over
 * its tokens in a paged K and a paged V pool.  For query head h, which reads
 * KV head h / (heads / kv_heads), and the request's attended tokens t:
 *     s_t = scale * q_h . k_t,   lse = ln sum_t e^(s_t),
 *     out_h = sum_t e^(s_t - lse) v_t.
 * Attended are tokens 0 .. lens[r] - 1; with window > 0, of those only the
 * first `sink` and the last `window` (the new token's own row, appended
 * before the call, is the last one).
 *   q            : DEVICE [R][q_ld], head h of request r at element
 *                  r * q_ld + h * head_dim; q_ld % 8 == 0, so q may be a
 *                  column slice of a fused projection's rows.
 *   k_cache, v_cache : DEVICE pools [num_blocks][16][kv_heads * head_dim].
 *   block_table  : DEVICE int32 [R][max_blocks], as for
 *                  kvtc_decompress_paged; requests may share blocks.
 *   lens         : DEVICE int32 [R] (negative counts as 0; above
 *                  16 * max_blocks it counts as that and flags
 *                  KVTC_FLAG_SPACE).
 *   scale        : at most 2^127 in magnitude, not NaN.  A product q_h . k_t
 *                  or s_t log2(e) beyond fp32's range counts as infinite.
 *   out          : DEVICE [R][out_ld], laid out as q; elements between the
 *                  rows are untouched.
 *   lse          : DEVICE fp32 [R][heads], or NULL: the log-sum-exp, with
 *                  which results over disjoint tokens can be joined.
 * q, the pools and out hold `dtype` elements (enum kvtc_dtype).  Tokens in
 * blocks whose id is outside [0, num_blocks) are left out and flag
 * KVTC_FLAG_BLOCK.  Rows of a block that are not attended may hold anything
 * (infinities and NaN included).  A head whose weights e^(s_t) sum to zero
 * (no attended token, or every s_t = -inf) gets out = 0, lse = -inf; a NaN
 * or s_t = +inf in the attended tokens gives NaN, an infinity in V an
 * infinity (or NaN, where its weight is below 2^-20).  Products are summed,
 * and the softmax statistics held, in fp32.  A weight enters its product with
 * v as two 16-bit terms, to 2^-15 of itself; exponentials and the reciprocal
 * of their sum are the hardware's approximate ones (2^-22); out is rounded
 * once.  Against fp32 weights that moves one value of out in a thousand in
 * bf16, three in fp16, to its neighbour; the error against 64 bits stays.  The
 * result does not depend on timing, so equal calls on one device give equal
 * bits.
 *   head_dim 64, 128 or 256; kv_heads * head_dim <= 8192; at most 128 query
 * heads a KV head; num_blocks < 2^31, max_blocks < 2^27 - 1.  out, lse and
 * workspace must not overlap an input or one another.
 * workspace: device scratch of kvtc_paged_attend_workspace_bytes bytes, used
 * only while the call's work runs on cuda_stream: calls that may run at the
 * same time need one each.  q, pools, out and workspace 16-byte aligned,
 * block_table, lens and lse 4.
 * Errors: EINVAL, ESIZE, EALIGN, ENOTSUP, ECUDA.
 */
int kvtc_paged_attend(int cuda_device, int R, int heads, int kv_heads,
                      int head_dim, int dtype, const void* q, int64_t q_ld,
                      const void* k_cache, const void* v_cache,
                      int64_t num_blocks, int block_size,
                      const int32_t* block_table, int max_blocks,
                      const int32_t* lens, int sink, int window, float scale,
                      void* out, int64_t out_ld, float* lse, void* workspace,
                      int64_t workspace_bytes, uint32_t* flags,
                      void* cuda_stream);

/*
 * Chunks of new tokens -- the calls around kvtc_paged_attend where a request
 * brings more than one new token at a time (a prompt, a piece of one, drafted
 * tokens), and the calls that shrink a cache to what attention weighs.  What
 * is said above of the paged serving calls (device, streams, graphs, flags,
 * blocks of 16 tokens, R <= 4096) holds for these too.  The rows of all
 * requests lie behind one another: those of request r are rows cu[r] ..
 * cu[r + 1] - 1 of N (cu as kvtc_paged_assign writes it: DEVICE int64
 * [R + 1], non-decreasing; values outside [0, N] count as the nearer end,
 * and above N flag KVTC_FLAG_SPACE), and belong to the last tokens of lens[r]:
 * row cu[r] + i of n is token lens[r] - n + i.  Rows of no request (a padded
 * batch) are not read, and what belongs to them is left as it is.
 */

/* How kvtc_rotary_frequencies stretches positions for long contexts. */
enum kvtc_rotary_scaling {
  KVTC_ROTARY_PLAIN = 0,   /* f_i = base^(-2 i / rotary_dim) */
  KVTC_ROTARY_LINEAR = 1,  /* f_i / factor: positions divided by factor */
  KVTC_ROTARY_BASE = 2,    /* base * factor^(rotary_dim / (rotary_dim - 2)):
                              the longest wavelength times factor, the
                              shortest as it is */
  KVTC_ROTARY_BANDS = 3    /* f_i (a + (1 - a) / factor), a from 0 to 1 as
                              the turns of f_i in `context` tokens go from
                              `low` to `high` */
};

/*
 * kvtc_rotary_frequencies -- angles per position for kvtc_paged_rotate, into
 * a HOST array of rotary_dim / 2 doubles (no device is touched).
 *   base    : > 0, finite.
 *   factor  : > 0, finite (not read for KVTC_ROTARY_PLAIN).
 *   context, low, high : for KVTC_ROTARY_BANDS alone: context > 0,
 *             0 <= low < high, all finite.
 * rotary_dim is even and positive (above 2 for KVTC_ROTARY_BASE).
 * Errors: EINVAL (where a frequency is not finite too; nothing is written then).
 */
int kvtc_rotary_frequencies(int rotary_dim, double base, int scaling,
                            double factor, double context, double low,
                            double high, double* inv_freq);

/*
 * kvtc_paged_rotate -- norms and rotary positions of N new tokens' queries
 * and keys, the queries into q_out, keys and values into the pools.  Each
 * head x of q (and of k):
 *     y = x / sqrt(mean(x^2) + eps) * norm            (y = x where norm is
 *                                                      NULL),
 *     (y_a, y_b) -> rotary_scale (y_a cos t - y_b sin t, y_b cos t + y_a sin t)
 * for the pairs i = 0 .. rotary_dim / 2 - 1, t = positions * inv_freq[i]; the
 * elements behind rotary_dim stay y.  Values v are copied bit for bit.
 *   q, k, v      : DEVICE rows of `dtype` elements, token n at n * ld: column
 *                  slices of one projection's rows, heads side by side.
 *                  v may be NULL with v_cache (keys alone).
 *   positions    : DEVICE int32 [N], any value.  May be NULL when rotary_dim
 *                  is 0.
 *   inv_freq     : DEVICE fp64 [rotary_dim / 2], finite, as
 *                  kvtc_rotary_frequencies gives them.  May be NULL when
 *                  rotary_dim is 0.
 *   rotary_dim   : % 8 == 0, 0 .. head_dim.
 *   interleaved  : 0: pair i is elements i and i + rotary_dim / 2; else
 *                  2 i and 2 i + 1.
 *   q_norm, k_norm : DEVICE [head_dim] of `dtype` each, or NULL.
 *   eps          : >= 0, finite.
 *   q_out        : DEVICE [N][q_out_ld] of `dtype`, every row written; may be
 *                  q itself with q_out_ld == ld.
 *   slots        : DEVICE int64 [N] and
 *   k_cache, v_cache : [num_blocks][16][kv_heads * head_dim], as for
 *                  kvtc_paged_append (slots outside skip the token's k and v;
 *                  above the pool they flag KVTC_FLAG_BLOCK).
 * All arithmetic is in fp32, rounded once; the angle is taken modulo a turn
 * in 64-bit fixed point, so it is as exact at far positions as at near ones
 * (to p 2^-53 of a turn of f_i at position p, through inv_freq / 2 pi, and
 * 2^-25 of a turn).
 *   head_dim 64, 128 or 256; kv_heads * head_dim <= 8192, heads * head_dim <=
 * 131072.  All pointers to rows, norms and pools 16-byte aligned, ld and
 * q_out_ld % 8 == 0, slots and inv_freq 8, positions 4.  Other than as said no
 * output may overlap an input or another output.  One kernel launch.
 * Errors: EINVAL, ESIZE, EALIGN, ENOTSUP, ECUDA.
 */
int kvtc_paged_rotate(int cuda_device, int64_t N, int heads, int kv_heads,
                      int head_dim, int dtype, const void* q, const void* k,
                      const void* v, int64_t ld, const int32_t* positions,
                      const double* inv_freq, int rotary_dim, int interleaved,
                      float rotary_scale, const void* q_norm,
                      const void* k_norm, float eps, void* q_out,
                      int64_t q_out_ld, const int64_t* slots, int block_size,
                      void* k_cache, void* v_cache, int64_t num_blocks,
                      uint32_t* flags, void* cuda_stream);

/* Device workspace bytes kvtc_paged_attend_chunks needs (< 0 on error). */
int64_t kvtc_paged_attend_chunks_workspace_bytes(int cuda_device, int R,
                                                 int64_t N, int heads,
                                                 int kv_heads, int head_dim);

/*
 * kvtc_paged_attend_chunks -- attention of chunks of new tokens over their
 * requests' tokens in the pools, the chunk's own among them (appended before
 * the call).  The row of token p attends to tokens 0 .. p; with window > 0, of
 * those only to the first `sink` and the last `window` (p is the last one):
 * what kvtc_paged_attend computes for lens = p + 1.  Formulas, layouts and the
 * meaning of q, k_cache, v_cache, block_table, lens, scale, out and lse are
 * kvtc_paged_attend's, with N rows (q [N][q_ld], out [N][out_ld], lse
 * [N][heads]) in the place of R.
 * A row whose token is before the first (more rows than lens[r]) and a head
 * whose weights sum to zero get out = 0, lse = -inf; tokens in blocks whose
 * id is out of range are left out and flag KVTC_FLAG_BLOCK.  Infinities and
 * NaN in K, V or q reach the rows that attend to them and no others (an
 * infinity in V as an infinity, or NaN where its weight is below 2^-20).
 * Products are summed, and the softmax statistics held, in fp32.  A weight
 * enters its product with v as one `dtype` number (half a step of it, relative;
 * in fp16 to 2^-32 of the largest weight at least), the sum of the weights is of
 * the unrounded ones; exponentials and the reciprocal of their sum are the
 * hardware's approximate ones (2^-22); out is rounded once.  Against 64 bits the
 * weights' rounding adds up to half a step of `dtype`, relative, of
 * sum_t e^(s_t - lse) |v_t| to the half step of out.  In the 2-norm the error is
 * that of out's own rounding, to a tenth, where V's mean outweighs its spread,
 * and 1.4 times that where V has no mean and many tokens share the weight
 * (kvtc_paged_attend, whose weights have two terms, stays at 1.0 there).  Equal
 * calls on one device give equal bits.
 *   head_dim 64, 128 or 256; kv_heads * head_dim <= 8192; at most 128 query
 * heads a KV head.  Alignment and overlap as for kvtc_paged_attend, cu 8.
 * workspace: device scratch of kvtc_paged_attend_chunks_workspace_bytes
 * bytes (20 to 41 MB), used only while the call's work runs on cuda_stream:
 * calls that may run at the same time need one each.  Two kernel launches; one
 * where the table has at most 64 columns (at head_dim 256 mostly 32) and there
 * are few rows.
 * Errors: EINVAL, ESIZE, EALIGN, ENOTSUP, ECUDA.
 */
int kvtc_paged_attend_chunks(
    int cuda_device, int R, int64_t N, int heads, int kv_heads, int head_dim,
    int dtype, const void* q, int64_t q_ld, const void* k_cache,
    const void* v_cache, int64_t num_blocks, int block_size,
    const int32_t* block_table, int max_blocks, const int64_t* cu,
    const int32_t* lens, int sink, int window, float scale, void* out,
    int64_t out_ld, float* lse, void* workspace, int64_t workspace_bytes,
    uint32_t* flags, void* cuda_stream);

/* Device workspace bytes kvtc_paged_weigh needs (< 0 on error). */
int64_t kvtc_paged_weigh_workspace_bytes(int cuda_device, int R, int64_t N,
                                         int heads, int kv_heads,
                                         int head_dim);

/*
 * kvtc_paged_weigh -- the attention weight that each cached token receives:
 *     acc_out[r][t] = decay acc[r][t] + sum e^(scale q_ih . k_t - lse_ih)
 * over request r's rows i that attend to t (as kvtc_paged_attend_chunks has
 * it) and all query heads h, for t < lens[r]; other elements of acc_out are
 * left as they are.
 *   lse          : DEVICE fp32 [N][heads], what the attention of the same
 *                  rows returned.  A head whose lse is -inf adds nothing.
 *   decay        : finite; where it is 0, acc is not read and may be NULL.
 *   acc, acc_out : DEVICE fp32 [R][acc_ld], acc_ld >= 16 * max_blocks,
 *                  % 4 == 0; acc_out may be acc itself.
 * The others are kvtc_paged_attend_chunks' (a few of its rows may be given,
 * with a cu of their own, if they are the requests' last).  Every row is
 * multiplied with every tile of 256 tokens that any row of its request attends
 * to, so the last rows of a prompt cost far less than all of them.  Tokens in
 * blocks whose id is out of range receive nothing and, where attended, flag
 * KVTC_FLAG_BLOCK.  Sums are in fp32, in a fixed order: equal calls on one
 * device give equal bits.  A weight is off, relative, by its score's error (a
 * sum of head_dim products in fp32) and by 2^-22 (1 + |lse|).  Two kernel
 * launches.  workspace: device scratch of
 * kvtc_paged_weigh_workspace_bytes bytes, used only while the call's work runs
 * on cuda_stream; calls that may run at the same time need one each.  No output
 * may overlap an input other than as said.  acc, acc_out, q, k_cache and
 * workspace 16-byte aligned, cu 8, the others 4.
 * Errors: EINVAL, ESIZE, EALIGN, ENOTSUP, ECUDA.
 */
int kvtc_paged_weigh(int cuda_device, int R, int64_t N, int heads,
                     int kv_heads, int head_dim, int dtype, const void* q,
                     int64_t q_ld, const void* k_cache, int64_t num_blocks,
                     int block_size, const int32_t* block_table,
                     int max_blocks, const int64_t* cu, const int32_t* lens,
                     int sink, int window, float scale, const float* lse,
                     float decay, const float* acc, float* acc_out,
                     int64_t acc_ld, void* workspace, int64_t workspace_bytes,
                     uint32_t* flags, void* cuda_stream);

/* Device workspace bytes kvtc_paged_evict needs (< 0 on error). */
int64_t kvtc_paged_evict_workspace_bytes(int R, int max_blocks);

/*
 * kvtc_paged_evict -- cut requests down to `keep` cached tokens.  Of a
 * request with more than `keep`, the first `sink`, the last `window` and, of
 * the others, the keep - sink - window with the greatest acc stay (of equal
 * ones those with the lowest index; -0 equals 0, a NaN is below -inf).  What
 * stays keeps its order and becomes tokens 0 .. lens_out[r] - 1.
 *   acc          : DEVICE fp32 [R][acc_ld] (as kvtc_paged_weigh's): a weight
 *                  per token.
 *   lens         : DEVICE int32 [R] (negative counts as 0; above 16 *
 *                  max_blocks as that, and flags KVTC_FLAG_SPACE).
 *   keep, sink, window : sink + window <= keep.
 *   block_table  : DEVICE int32 [R][max_blocks]: the blocks that tokens are
 *                  in.
 *   out_table    : the blocks that they go to, laid out the same.  Either
 *                  block_table itself (the call works in place, and the
 *                  request's blocks must be its own), or a table none of
 *                  whose blocks that are written to is read from in this
 *                  call.  Its columns ceil(lens_out[r] / 16) and up are not
 *                  read; giving blocks back is the caller's.
 *   cache        : HOST array [nstreams] of pools [num_blocks][16][D] of
 *                  16-bit elements (any number of layers' K and V that share
 *                  the tables); D % 8 == 0, at most 8192.
 *   kept         : DEVICE int32 [R][keep], written whole: where token j was,
 *                  -1 from lens_out[r] on.  May be NULL when keep is 0.
 *   acc_out      : DEVICE fp32 [R][acc_ld]: the weights of what stays, then
 *                  zeros up to lens[r]; may be acc itself.
 *   lens_out     : DEVICE int32 [R], written: min(lens[r], keep); may be lens
 *                  itself.
 * A token whose old or new block id is out of range stays in the list, its
 * rows are not written, and KVTC_FLAG_BLOCK is set (new ids are looked at where
 * there are pools).  workspace: device scratch
 * of kvtc_paged_evict_workspace_bytes bytes (8 for each token that the table
 * has place for), used only while the call's work runs on cuda_stream; calls
 * that may run at the same time need one each.  One kernel launch, and one per
 * 64 pools.  cache, acc, acc_out and workspace 16-byte aligned, acc_ld % 4 ==
 * 0, the others 4.  Other than as said no output may overlap an input or
 * another output.
 * Errors: EINVAL, ESIZE, EALIGN, ENOTSUP, ECUDA.
 */
int kvtc_paged_evict(int cuda_device, int R, const float* acc, int64_t acc_ld,
                     const int32_t* lens, int keep, int sink, int window,
                     const int32_t* block_table, const int32_t* out_table,
                     int max_blocks, int block_size, int nstreams,
                     void* const* cache, int D, int64_t num_blocks,
                     int32_t* kept, float* acc_out, int32_t* lens_out,
                     void* workspace, int64_t workspace_bytes,
                     uint32_t* flags, void* cuda_stream);

/*
 * kvtc_calibrate -- the one-time calibration of technical summary 2A, on
 * the GPU, writing a version-1 blob (format above).  Per stream: mu = mean of
 * the calibration rows; V = eigenvectors of their covariance, sorted by
 * eigenvalue descending, each signed so that its largest-magnitude entry is
 * positive; E[g][b] = summed squared coefficient error of group g at width
 * b (b = 0: the group's energy) measured with the codec's quantiser; widths
 * = the DP allocation minimising sum E[g][b_g] with sum (32 + 16 b_g) over
 * groups with b_g > 0 at most budget_bits (ties keep the smaller width).
 *   tokens      : HOST array [n] of device pointers, stream i's calibration
 *                 rows, bf16 [N][ld]; layers, kvs: HOST arrays [n].
 *   blob        : HOST output of capacity bytes (kvtc_blob_max_bytes is an
 *                 upper bound); *blob_bytes receives the size (also when
 *                 the capacity is too small: ESIZE).
 * Unlike the codec calls it allocates temporary device memory (freed before
 * returning) and synchronises cuda_stream.  fp64 arithmetic on the device:
 * mean, covariance, eigenvector order and signs, coefficient products,
 * distortion table and DP are this library's kernels; the symmetric
 * eigensolver is cuSOLVER's (syevd).
 * Errors: EINVAL, ENOMEM, ECUDA, ESIZE.
 */
int kvtc_calibrate(int cuda_device, int n, const int* layers, const int* kvs,
                   const void* const* tokens, int64_t N, int64_t ld, int D,
                   int sink, int window, int budget_bits, void* blob,
                   size_t capacity, size_t* blob_bytes, void* cuda_stream);

/* Upper bound on the blob size of n streams of width D (< 0 on error). */
int64_t kvtc_blob_max_bytes(int n, int D);

/* Synchronise cuda_stream, then return the sticky device flags in *flags
 * (KVTC_FLAG_*) and clear them.  Returns KVTC_OK or ECUDA. */
int kvtc_device_status(const kvtc_calib* calib, void* cuda_stream,
                       unsigned* flags);

/*
 * kvtc_wait_selftest -- exercise the bounded wait that every kernel of this
 * library uses on its mbarriers (the pages have no counterpart: this is a
 * failure-detection check).  One thread waits, for at most limit_us
 * microseconds, on a barrier that nothing ever arrives at; when the limit
 * runs out it sets KVTC_FLAG_TIMEOUT in the handle's sticky flag word, the
 * same way a kernel reports a wait that ran out, and returns.  Read the
 * flag with kvtc_device_status; the context stays usable.
 *   limit_us    : 1 .. 2000000.
 *   cuda_stream : the launch is enqueued on it.
 * Errors: EINVAL, ECUDA.
 */
int kvtc_wait_selftest(const kvtc_calib* calib, uint32_t limit_us,
                       void* cuda_stream);

/*
 * kvtc_calib_mean_static -- the per-channel mean of calibration rows (the
 * mean that kvtc_calibrate stores for a stream), computed without
 * allocating any device memory.  The paper has no counterpart: this entry
 * point exists for callers that cannot call cudaMalloc, such as serving
 * engines that give nearly all device memory to their own KV-cache pool at
 * start-up, or latency-sensitive paths that cannot take the device-wide
 * synchronisation of cudaMalloc / cudaFree.
 *   tokens : device bf16 rows [N][ld] (N >= 1, ld >= D).
 *   mu_out : device fp64 [D], written.
 *   D      : at most 4096; wider rows return KVTC_ESIZE.
 * Scratch comes from a fixed 1 MiB array inside the library.  CUDA loads
 * modules lazily by default, so the array comes into being on a device at
 * the first call there, which loads this code and looks up the array's
 * device address (a one-time set-up), and it is then held until the process
 * exits.  That first call can therefore fail with ECUDA when the device has
 * no free memory left: make it before reserving the device's memory for a
 * KV pool (or run with CUDA_MODULE_LOADING=EAGER, which creates the array
 * with the context), and before any stream capture.  All calls on a device
 * share the array: each call writes every entry it reads, but calls that
 * overlap on the GPU race with each other, so serialise them.  No
 * cudaMalloc, cudaFree or allocating library routine is called.  Enqueued
 * on cuda_stream.
 * Errors: EINVAL, ESIZE, ECUDA.
 */
int kvtc_calib_mean_static(int cuda_device, const void* tokens, int64_t N,
                           int64_t ld, int D, double* mu_out,
                           void* cuda_stream);

/* Number of kernels this library has launched since it was loaded (all
 * devices and threads); a cheap way for callers to count launches. */
uint64_t kvtc_launch_count(void);

/* Static description of a status code. */
const char* kvtc_strerror(int status);

#ifdef __cplusplus
}
#endif
#endif /* KVTC_H */
