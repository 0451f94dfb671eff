/*
 * splitzip.h -- C ABI of the MI355X (gfx950) SplitZip BF16 KV-cache codec.
 *
 * The method is the one the SplitZip explainers describe ("SplitZip: Ultra
 * Fast Lossless KV Compression for Disaggregated LLM Serving", gist.science
 * pages for arXiv 2605.01708, French and Japanese): every BF16 word is split
 * into sign, exponent and mantissa (section "1. La structure de la Note");
 * the 16 most frequent exponents of the tensor get fixed 4-bit codes, two
 * codes per byte, and every other exponent is written as a (position,
 * exponent) escape record (section "3. La strategie SplitZip"); decoding
 * looks the codes up, recombines them with sign and mantissa and overwrites
 * the escaped slots (section "4. Pourquoi est-ce rapide ?"); the round trip
 * is bit-exact (section "Les Resultats").
 *
 * Container produced by sz_encode (little-endian, no padding):
 *   off 0    u32  magic 0x564B5A53 (bytes 'S' 'Z' 'K' 'V')
 *   off 4    u16  version 1
 *   off 6    u16  element type 1 (bf16)
 *   off 8    u64  N, number of elements
 *   off 16   u64  E, number of escapes
 *   off 24   u64  total bytes = 176 + ceil(N/2) + N + 5E
 *   off 32   u64  seg_end[16]: number of escapes whose position is below
 *                 (s+1) * 2^32 (escape positions are stored modulo 2^32)
 *   off 160  u8   codebook[16]: code c -> exponent; codes are ranks by count
 *                 (descending), equal counts ordered by exponent (ascending)
 *   off 176  u8   nibbles[ceil(N/2)]: element 2j in the low nibble of byte j,
 *                 element 2j+1 in the high nibble; escaped elements hold 0
 *   +        u8   sm[N]: sign in bit 7, mantissa in bits 6..0
 *   +        u32  pos_lo[E]: escape positions mod 2^32, strictly ascending
 *   +        u8   exp[E]: the exponent of each escape
 *
 * Conventions for every call below:
 *   - Pointers named d_* are device pointers (hipMalloc or a PyTorch CUDA
 *     tensor) owned by the caller; the library keeps none of them after the
 *     stream work completes.  BF16 and container pointers must be 16-byte
 *     aligned; workspaces 256-byte aligned.
 *   - Calls are asynchronous on `stream` and never synchronise the host,
 *     except the two sz_ship_* calls, which return when their data is in
 *     place.  The return value reports errors found on the host before
 *     anything is launched (nothing is launched then), or SZ_ERR_HIP for a
 *     failed launch or allocation.  Results are valid once the stream work
 *     is done.
 *   - Calls on different streams may run concurrently if they use different
 *     buffers.
 */
#ifndef SPLITZIP_H
#define SPLITZIP_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SZ_HEADER_BYTES 160u
#define SZ_CODEBOOK_BYTES 16u
#define SZ_PREFIX_BYTES 176u
#define SZ_MAX_ELEMENTS (1ull << 36)

typedef enum {
    SZ_OK = 0,
    SZ_ERR_INVALID_ARGUMENT = 1, /* NULL or misaligned pointer, overlap, bad workspace */
    SZ_ERR_CAPACITY = 2,         /* destination smaller than sz_max_compressed_size(n) */
    SZ_ERR_TOO_LARGE = 3,        /* n > SZ_MAX_ELEMENTS */
    SZ_ERR_CORRUPT = 4,          /* container inconsistent with n or with itself */
    SZ_ERR_HIP = 5               /* a HIP launch or allocation failed */
} sz_status;

/* Upper bound of the container size for n elements: 176 + ceil(n/2) + n +
 * 5*floor(15n/16).  SplitZip explainer section "3. La strategie SplitZip":
 * every exponent gets a fixed 4-bit code stored two per byte (ceil(n/2)
 * bytes), every word keeps its sign and mantissa (n bytes), and an exponent
 * outside the 16-entry list costs one (position, exponent) note (5 bytes
 * here); the 16 most frequent of 256 exponents always cover at least n/16
 * elements, so at most floor(15n/16) words need a note.  Returns 0 when
 * n > SZ_MAX_ELEMENTS.  Host-only, touches no device. */
uint64_t sz_max_compressed_size(uint64_t n_elements);

/* Bytes of device workspace the staged encode calls need for n elements
 * (at most about 4.3 MB).  Host-only. */
uint64_t sz_workspace_size(uint64_t n_elements);

/* Compress n BF16 words at d_src into the container format above at d_dst.
 * SplitZip explainer section "3. La strategie SplitZip" (top-16 exponent
 * codebook, 4-bit codes two per byte, escape records for the rest).
 *   d_src             n little-endian BF16 words (any bit patterns)
 *   d_dst             container buffer, dst_capacity bytes; must be at least
 *                     sz_max_compressed_size(n) (else SZ_ERR_CAPACITY).  The
 *                     container is its first `total bytes`; any byte below
 *                     sz_max_compressed_size(n) may be written (see below),
 *                     none at or past it
 *   d_compressed_size optional device u64 that receives the container size
 *                     (the same value is stored at container offset 24)
 * From 2^26 elements on (sz_encode_single_read(n) says 1) the input is read
 * once when a sample of it predicts the codebook: the bytes of d_dst past the
 * container, up to sz_max_compressed_size(n), then serve as scratch and are
 * left unspecified.  The container is the same either way.
 * Allocates its workspace (sz_workspace_size(n)) from a library-owned,
 * stream-ordered device memory pool and returns it on the same stream.
 * While `stream` is being captured into a graph, returns
 * SZ_ERR_INVALID_ARGUMENT and launches nothing: the staged calls below, with
 * a workspace the caller owns, are the capturable form. */
sz_status sz_encode(const void *d_src, uint64_t n_elements, void *d_dst,
                    uint64_t dst_capacity, uint64_t *d_compressed_size,
                    hipStream_t stream);

/* For callers that cannot allocate device memory (code under graph
 * capture, tight serving loops, harnesses that forbid allocation):
 * sz_encode with the same arguments, passes and container, but its
 * workspace is a fixed array of SZ_NOALLOC_WORKSPACE_BYTES in the library's
 * device memory, one per GPU, loaded with the library and held until the
 * process ends.  The call allocates nothing (no hipMalloc, no pool, no
 * hipFree) and may be captured into a graph.  Every call on one GPU uses
 * that GPU's array: calls that can overlap on one GPU (other streams, or
 * several replays of graphs in flight at once) race and give unspecified
 * containers, so callers serialise them.  No pass needs the array to hold
 * anything at its start (each pass writes what the next one reads).
 * SZ_ERR_TOO_LARGE when n's workspace (sz_workspace_size(n)) exceeds the
 * array; with this library's chunk plan no n up to SZ_MAX_ELEMENTS does. */
#define SZ_NOALLOC_WORKSPACE_BYTES (4608ull * 1024ull)
sz_status sz_encode_noalloc(const void *d_src, uint64_t n_elements, void *d_dst,
                            uint64_t dst_capacity, uint64_t *d_compressed_size,
                            hipStream_t stream);

/* Decompress a container of src_bytes bytes into n BF16 words at d_dst,
 * bit-exactly.  SplitZip explainer section "4. Pourquoi est-ce rapide ?"
 * (code -> exponent lookup, recombination with sign and mantissa, escaped
 * slots overwritten).  The form depends on the size and escape density:
 * from 2^26 words with at most one escape in 128, one pass over grid-stride
 * tiles (sz_decode_index, then sz_decode_tiles, with a workspace from a
 * library-owned stream-ordered pool); below 2^26 words with at most one
 * escape in 256, the two passes sz_decode_unpack and sz_decode_scatter;
 * otherwise, and whenever the stream is being captured into a graph, one
 * pass with a per-word exponent map (sz_decode_dense).  Same result every
 * way.
 *   src_bytes   must equal the container's total size: the host derives E
 *               from it, so no device read is needed before launching
 *   d_status    optional device i32: SZ_OK, or SZ_ERR_CORRUPT when the
 *               header or an escape position fails a check on the device
 *               (d_dst content is then unspecified, but no write ever leaves
 *               d_dst[0..n))
 * Host-side SZ_ERR_CORRUPT: src_bytes < 176 + ceil(n/2) + n, or the rest is
 * not a multiple of 5 bytes, or implies more than floor(15n/16) escapes. */
sz_status sz_decode(const void *d_src, uint64_t src_bytes, void *d_dst,
                    uint64_t n_elements, int32_t *d_status, hipStream_t stream);

/* ---- staged form: the same kernels, one call per pass ------------------
 * sz_encode = sz_encode_histogram; sz_encode_codebook; sz_encode_pack on one
 * stream with one workspace of at least sz_workspace_size(n) bytes that the
 * caller owns and does not touch in between.  sz_decode_unpack followed by
 * sz_decode_scatter gives the same words and status as sz_decode.
 * Out-of-order use cannot write outside the caller's buffers, but yields an
 * unspecified result. */

/* Pass 1, exponent histogram (explainer section "2. La decouverte
 * secrete": the exponents are highly repetitive): one 256-bin count per
 * fixed-size chunk of the input, into the workspace. */
sz_status sz_encode_histogram(const void *d_src, uint64_t n_elements,
                              void *d_workspace, uint64_t workspace_bytes,
                              hipStream_t stream);

/* Pass 2, top-16 selection (section "3. La strategie SplitZip", shortcut
 * bullet): merges the chunk counts, ranks the 256 exponents, writes the
 * header and codebook to d_dst, the escape offset of every chunk to the
 * workspace and the container size to *d_compressed_size (optional). */
sz_status sz_encode_codebook(uint64_t n_elements, void *d_workspace,
                             uint64_t workspace_bytes, void *d_dst,
                             uint64_t dst_capacity, uint64_t *d_compressed_size,
                             hipStream_t stream);

/* Pass 3, packing (same section, packing and rare-value bullets): 4-bit
 * codes two per byte, sign|mantissa bytes, and the escape records of each
 * chunk written to their final slots in ascending position order. */
sz_status sz_encode_pack(const void *d_src, uint64_t n_elements,
                         const void *d_workspace, uint64_t workspace_bytes,
                         void *d_dst, uint64_t dst_capacity, hipStream_t stream);

/* Passes 2 and 3 in one launch, after sz_encode_histogram, for
 * 1 <= n_elements <= 2^21 (at most 128 chunks of the plan; otherwise
 * SZ_ERR_INVALID_ARGUMENT): every pack workgroup sums and ranks the chunk
 * counts itself (the selection of section "3. La strategie SplitZip") and
 * works out its chunk's first escape slot, so no codebook pass runs between
 * the two launches.  Writes the same container as sz_encode_codebook then
 * sz_encode_pack, and the container size to *d_compressed_size (optional);
 * sz_encode takes this form for such n.  Same arguments and checks as
 * sz_encode_pack. */
sz_status sz_encode_pack_ranked(const void *d_src, uint64_t n_elements,
                                const void *d_workspace, uint64_t workspace_bytes,
                                void *d_dst, uint64_t dst_capacity,
                                uint64_t *d_compressed_size, hipStream_t stream);

/* ---- staged form of the single-read encode (n >= 2^20) -----------------
 * sz_encode_sample; sz_encode_first_pass; sz_encode_finish on one stream,
 * one workspace, gives the container of sz_encode.  Not part of the pages'
 * method: a way to read the input once.  A fixed sample (512 blocks of 2048
 * words spread evenly over the input) gives a provisional codebook by the
 * same ranking rule; the first pass packs every chunk with it while it
 * takes the exact counts; the finish pass ranks the exact codebook, then
 * keeps what the first pass wrote when the exact codebook equals the
 * provisional one, rewrites the 4-bit codes when it holds the same 16
 * exponents in another order, and packs again (a second read) otherwise,
 * or when a chunk held more than 1/16 escapes, or when the sample predicted
 * more than one escape in 32.  The workspace may hold any bytes before the
 * first call: every call gives the same container (the first call on a
 * workspace in an unknown state may take the slower finish).
 * These calls return SZ_ERR_INVALID_ARGUMENT for n < 2^20 (besides the
 * checks of the two-read calls); the first pass and the finish use the bytes
 * of d_dst past the container, up to sz_max_compressed_size(n), as scratch. */

/* 1 when sz_encode takes the single-read passes for n elements (n >= 2^26),
 * else 0.  Host-only. */
int sz_encode_single_read(uint64_t n_elements);

/* The sample's exponent counts, then the provisional codebook and whether
 * the first pass packs, into the workspace. */
sz_status sz_encode_sample(const void *d_src, uint64_t n_elements, void *d_workspace,
                           uint64_t workspace_bytes, hipStream_t stream);

/* The first pass: the exact per-chunk exponent counts to the workspace (laid
 * out for sz_encode_finish, not for sz_encode_codebook) and, when the sample
 * predicts few escapes, the nibble and sign|mantissa streams plus each
 * chunk's escape records (to the scratch area). */
sz_status sz_encode_first_pass(const void *d_src, uint64_t n_elements,
                               void *d_workspace, uint64_t workspace_bytes,
                               void *d_dst, uint64_t dst_capacity, hipStream_t stream);

/* The exact codebook (the selection of section "3. La strategie SplitZip",
 * as sz_encode_codebook takes it), the header, and the container size to
 * *d_compressed_size (optional); then escape records to their final slots,
 * codes rewritten, or the input packed again, as described above. */
sz_status sz_encode_finish(const void *d_src, uint64_t n_elements,
                           void *d_workspace, uint64_t workspace_bytes,
                           void *d_dst, uint64_t dst_capacity,
                           uint64_t *d_compressed_size, hipStream_t stream);

/* Decode pass 1: header check (sets *d_status to SZ_OK or SZ_ERR_CORRUPT)
 * and every word rebuilt from its code and its sign|mantissa byte. */
sz_status sz_decode_unpack(const void *d_src, uint64_t src_bytes, void *d_dst,
                           uint64_t n_elements, int32_t *d_status,
                           hipStream_t stream);

/* Decode pass 2: every escape record overwrites the exponent field of the
 * word pass 1 wrote at its position; a position >= n or not above the
 * previous one raises *d_status to SZ_ERR_CORRUPT and is skipped.  Launches
 * nothing when E = 0. */
sz_status sz_decode_scatter(const void *d_src, uint64_t src_bytes, void *d_dst,
                            uint64_t n_elements, int32_t *d_status,
                            hipStream_t stream);

/* Decode in a single pass whatever the escape density: each workgroup
 * finds its range's escape records by a 64-way search over the sorted
 * positions, stages them in LDS and overwrites the escaped exponents before
 * the words are stored (explainer section "4. Pourquoi est-ce rapide ?").
 * Same arguments, result and status as sz_decode. */
sz_status sz_decode_fused(const void *d_src, uint64_t src_bytes, void *d_dst,
                          uint64_t n_elements, int32_t *d_status, hipStream_t stream);

/* Decode in a single pass, laid out for many escapes: each workgroup walks
 * its range in sub-ranges of 16384 words, reads the escape records of each
 * sub-range straight from the escape stream into a per-word LDS map, and
 * rebuilds the words with the mapped exponents in place of the codebook's
 * (explainer section "4. Pourquoi est-ce rapide ?").  Same arguments,
 * result and status as sz_decode, which picks this form above one escape
 * in 128 words, for small tensors above one in 256, and whenever it cannot
 * allocate. */
sz_status sz_decode_dense(const void *d_src, uint64_t src_bytes, void *d_dst,
                          uint64_t n_elements, int32_t *d_status, hipStream_t stream);

/* Decode in a single pass, one short-lived workgroup per 2048-word tile, in
 * two calls over a caller workspace of sz_decode_workspace_size(n) bytes
 * (256-byte aligned, not overlapping the container or the output; about
 * 72 bytes per tile plus 4 bytes per 64 possible escapes, at most 4 MiB of
 * those).  sz_decode_index
 * records, for every tile, the first escape record at or after the tile's
 * start and the tile's first records (each of its waves takes a run of 64
 * records and fills the tile entries up to its last record: no search), and
 * checks the header and that
 * the records ascend below n; sz_decode_tiles then rebuilds every tile's
 * words with its records' exponents in place of the codebook's (explainer
 * section "4. Pourquoi est-ce rapide ?").  sz_decode_tiles writes
 * *d_status (optional): SZ_OK, or SZ_ERR_CORRUPT when the index call found
 * a fault (the output content is then unspecified, but no write leaves
 * d_dst[0..n)); it only reads the workspace, so it may run again on the
 * same index.  The index call also copies each tile's records (up to 15)
 * into a 64-byte slot of the tile, which the tile call reads together with
 * the tile's codes; a tile with more records reads them from the escape
 * stream.  Together they give the result and status of sz_decode, which
 * takes this form, with a workspace from its pool, from 2^26 words with up
 * to one escape in 128. */
uint64_t sz_decode_workspace_size(uint64_t n_elements);
sz_status sz_decode_index(const void *d_src, uint64_t src_bytes, uint64_t n_elements,
                          void *d_workspace, uint64_t workspace_bytes, hipStream_t stream);
sz_status sz_decode_tiles(const void *d_src, uint64_t src_bytes, const void *d_workspace,
                          uint64_t workspace_bytes, void *d_dst, uint64_t n_elements,
                          int32_t *d_status, hipStream_t stream);

/* ---- paged tensors -----------------------------------------------------
 * Serving stacks keep KV caches in fixed-size pages (the explainers'
 * serving setting, section "Les Resultats").  These calls take such a
 * tensor as it lies: n words spread over pages of page_elems words, page i
 * at the device address d_pages[i] (d_pages is a device array of
 * pointers), so that the tensor is the concatenation of the pages in table
 * order (the last page may be partly used).  The container is exactly the
 * one sz_encode gives for that concatenation, so any decode call reads it,
 * and sz_decode_pages decodes any container into pages.  One launch per
 * pass for the whole tensor, whatever the number of pages.
 *   page_elems  a power of two, at least 16384
 *   n_pages     entries in d_pages; only the first ceil(n / page_elems)
 *               are read, each must be non-NULL and 16-byte aligned
 * The table's addresses are checked on the device: a NULL or misaligned
 * one makes the call touch no page and report SZ_ERR_INVALID_ARGUMENT in
 * *d_status (the container is then not valid).  Pages must not overlap
 * each other or the container.  The library allocates a small flag from
 * its stream-ordered pool (and, for encode, sz_encode's workspace), so
 * while `stream` is being captured into a graph both calls return
 * SZ_ERR_INVALID_ARGUMENT and launch nothing. */

/* sz_encode_pages: sz_encode of the paged tensor; *d_status (optional
 * device i32) receives SZ_OK or SZ_ERR_INVALID_ARGUMENT. */
sz_status sz_encode_pages(const void *const *d_pages, uint64_t n_pages, uint64_t page_elems,
                          uint64_t n_elements, void *d_dst, uint64_t dst_capacity,
                          uint64_t *d_compressed_size, int32_t *d_status, hipStream_t stream);

/* sz_decode_pages: sz_decode into the paged tensor (same forms, same
 * checks and status; SZ_ERR_INVALID_ARGUMENT in *d_status for a bad
 * page table). */
sz_status sz_decode_pages(const void *d_src, uint64_t src_bytes, void *const *d_pages,
                          uint64_t n_pages, uint64_t page_elems, uint64_t n_elements,
                          int32_t *d_status, hipStream_t stream);

/* ---- per-layer blocks, one container each -----------------------------
 * A serving stack holds a model's KV cache as one block per layer (the
 * explainers' serving setting, section "Les Resultats"), and each block may
 * travel on its own.  These calls take n_blocks blocks of block_elems words
 * each, block b at the device address d_blocks[b] (a device array of
 * pointers, each non-NULL and 16-byte aligned), and give block b its own
 * container, exactly the one sz_encode gives for that block alone, so that
 * sz_decode reads it too.  One launch per pass for all blocks.
 *   containers  block b's container starts at the container buffer plus
 *               b * pitch bytes (the buffer spans n_blocks * pitch bytes)
 *   d_sizes     device array of n_blocks u64: block b's container size
 *   n_blocks    1 .. 65535
 * Block addresses are checked on the device: a NULL or misaligned one
 * makes the calls touch none of that block's memory and report
 * SZ_ERR_INVALID_ARGUMENT as the block's status; the other blocks are
 * unaffected.  Blocks must not overlap one another or the containers.
 * Neither call allocates, so both may be captured into a graph.
 *
 * sz_blocks_workspace_size: bytes of device workspace sz_encode_blocks
 * needs: for each block, the per-chunk counts and escape bases of a chunk
 * plan made for all the blocks' words together (at most about 4.3 MB a
 * block, much less for small blocks), at 256-byte strides, then a flag
 * word per block; 0 for block_elems > SZ_MAX_ELEMENTS or a block count
 * outside 1 .. 65535.  Host-only. */
uint64_t sz_blocks_workspace_size(uint64_t block_elems, uint64_t n_blocks);

/* sz_encode_blocks: sz_encode of every block, each pass one launch for
 * all blocks, after an address check.  The passes are the ones sz_encode
 * takes for as many words as all blocks hold: from 2^26 words in total,
 * with blocks of at least 2^20 words, the single-read passes (sample,
 * first pass, finish), else the two-read ones (counts, codebook, pack).
 *   d_dst      container buffer, 16-byte aligned; dst_pitch a multiple of
 *              16 and at least sz_max_compressed_size(block_elems), else
 *              SZ_ERR_CAPACITY.  In the single-read form the bytes of a
 *              block's pitch past its container, up to
 *              sz_max_compressed_size(block_elems), serve as scratch and are
 *              left unspecified; no byte past that is written.
 *   d_sizes    written: each block's container size (0 for a block whose
 *              address failed the check)
 *   d_workspace, workspace_bytes   256-byte aligned, at least
 *              sz_blocks_workspace_size(block_elems, n_blocks); it may hold
 *              any bytes when the call starts
 *   d_status   optional device array of n_blocks i32: SZ_OK or
 *              SZ_ERR_INVALID_ARGUMENT per block */
sz_status sz_encode_blocks(const void *const *d_blocks, uint64_t n_blocks, uint64_t block_elems,
                           void *d_dst, uint64_t dst_pitch, uint64_t *d_sizes,
                           void *d_workspace, uint64_t workspace_bytes, int32_t *d_status,
                           hipStream_t stream);

/* sz_blocks_decode_workspace_size: bytes of device workspace that give
 * sz_decode_blocks its tile form (per block: a tile index, a fault flag
 * per 16384 words (64 to 4096 of them) and the tiles' record slots, at
 * 256-byte strides; about 1/30 of the block's words in bytes); 0 for bad
 * arguments as above.  Host-only. */
uint64_t sz_blocks_decode_workspace_size(uint64_t block_elems, uint64_t n_blocks);

/* sz_decode_blocks: the reverse, block b's container read from d_src +
 * b * src_pitch, d_sizes[b] bytes, and its words written to d_blocks[b],
 * with the checks of sz_decode.  A size that is no container of
 * block_elems words, or exceeds src_pitch, counts as corrupt: nothing
 * outside the block's pitch is read, and its words are then unspecified.
 * With d_workspace NULL, one pass per range of each block
 * (sz_decode_dense's form, the one for escape-heavy data); with a
 * workspace of at least sz_blocks_decode_workspace_size(block_elems,
 * n_blocks) bytes (256-byte aligned, any content), a tile index of every
 * block, then its tiles (sz_decode_index / sz_decode_tiles' form, the
 * faster one for KV data, and much the slower one at many escapes per
 * 2048 words).  Both forms are one launch per pass for all blocks.
 *   src_pitch  a multiple of 16, at least 176 + ceil(n/2) + n for
 *              n = block_elems
 *   d_status   required device array of n_blocks i32: SZ_OK, SZ_ERR_CORRUPT
 *              or SZ_ERR_INVALID_ARGUMENT per block */
sz_status sz_decode_blocks(const void *d_src, uint64_t src_pitch, const uint64_t *d_sizes,
                           uint64_t n_blocks, uint64_t block_elems, void *const *d_blocks,
                           void *d_workspace, uint64_t workspace_bytes, int32_t *d_status,
                           hipStream_t stream);

/* ---- operators on a paged cache ----------------------------------------
 * What a server does with the pages of a BF16 KV cache besides shipping
 * them (sz_encode_pages, sz_decode_pages): it puts the keys and values of
 * new tokens into them and attends over them.  Not part of the explainers'
 * method.  The calls below take one layer; they allocate nothing, never
 * synchronise and may be captured into a graph.  `stream` must belong to
 * the current device (SZ_ERR_INVALID_ARGUMENT otherwise).
 *
 * A head row is head_dim consecutive elements; head_dim is a multiple of 8,
 * 8 .. 256.  Tensors of rows are described by sz_heads.  A tensor that a
 * call writes must not overlap itself (rows lie inside one another's
 * strides: tokens of heads, or heads of tokens) nor any other tensor of the
 * call; two tensors may interleave with the same token stride, or with the
 * same token and head strides (slices of one fused projection).
 * sz_qk_norm_rope and sz_kv_append may write a BF16 tensor in place: same
 * data, strides and type as its source. */
typedef enum {
    SZ_TYPE_BF16 = 1,
    SZ_TYPE_F32 = 2
} sz_type;

typedef struct {
    void *data;            /* device address of token 0, head 0; 16-byte aligned */
    uint64_t heads;        /* 1 .. 65535 */
    uint64_t token_stride; /* elements from a token to the next; a multiple of 8, < 2^32 */
    uint64_t head_stride;  /* elements from a head to the next; a multiple of 8, < 2^32 */
    uint32_t type;         /* sz_type */
} sz_heads;

/* One layer's cache.  Sequence s keeps cached token c in page c /
 * page_tokens of its row of the tables, d_k_pages[s * table_pitch + c /
 * page_tokens] and the same of d_v_pages (device arrays of device
 * addresses, 16-byte aligned), at element (c mod page_tokens) *
 * token_stride + head * head_stride of the page.  With token_stride =
 * kv_heads * head_dim and head_stride = head_dim a sequence's pages in
 * table order are the tensor that sz_encode_pages reads.  A page spans
 * (page_tokens - 1) * token_stride + (kv_heads - 1) * head_stride +
 * head_dim BF16 words.  Table entries past a sequence's length, and those
 * that no token of a call needs, are never used and may hold anything.
 * Pages may be shared between sequences except where a call writes. */
typedef struct {
    const void *const *d_k_pages;
    const void *const *d_v_pages;
    uint64_t pages_per_seq; /* entries of a table row that may be used, >= 1 */
    uint64_t table_pitch;   /* entries from a row to the next, >= pages_per_seq */
    uint64_t token_stride;  /* elements; multiples of 8, below 2^26 and 2^32; */
    uint64_t head_stride;   /* rows must not overlap */
    uint32_t kv_heads;      /* 1 .. 65535 */
    uint32_t head_dim;
    uint32_t page_tokens;   /* a power of two, 16 .. 65536 */
} sz_kv_cache;

/* A ragged batch.  Sequence s has the new tokens d_starts[s] ..
 * d_starts[s+1] - 1 of the call's token-major tensors, and d_lens[s]
 * tokens in the cache, the new ones (its last) included.  Tokens before
 * d_starts[0] and from d_starts[n_seqs] on belong to no sequence and are
 * left as they are.  Both arrays are checked on the device. */
typedef struct {
    const int32_t *d_starts; /* n_seqs + 1 entries, ascending, 0 .. n_tokens */
    const int32_t *d_lens;   /* n_seqs entries, 0 .. pages_per_seq * page_tokens or 2^30 */
    uint64_t n_seqs;         /* 0 .. 65535 */
    uint64_t n_tokens;       /* rows of the token-major tensors, < 2^31 */
} sz_batch;

/* Rotation of positions over the first rotary_dim elements of a head:
 * pair i of rotary_dim / 2 turns by position * d_phases[i] / 2^64 turns,
 * and cos and sin are multiplied by `magnitude`.  The product is taken
 * modulo 2^64, so that no position loses accuracy. */
typedef struct {
    const uint64_t *d_phases; /* rotary_dim / 2 entries (sz_rope_phases) */
    uint32_t rotary_dim;      /* a multiple of 8, 0 (no rotation) .. head_dim */
    uint32_t interleaved;     /* 0: pair i is elements i, i + rotary_dim/2; 1: 2i, 2i + 1 */
    float magnitude;
} sz_rope;

/* How sz_rope_frequencies stretches the frequencies f_i = base^(-2i/R),
 * i < R/2, R = rotary_dim, by factor >= 1:
 *  PLAIN   f_i
 *  LINEAR  f_i / factor (position interpolation)
 *  BASE    base becomes base * factor^(R/(R-2)) (R > 2)
 *  RAMP    f_i where pair i turns more than `fast` times in original_len
 *          positions, f_i / factor where fewer than `slow` times, and
 *          between them a blend linear in i, from floor(i(fast)) to
 *          ceil(i(slow)), i(t) = R ln(original_len / (2 pi t)) / (2 ln base);
 *          *magnitude = 0.1 ln(factor) + 1 (YaRN)
 *  BANDS   the same ends, and between them a blend linear in the turns */
typedef enum {
    SZ_ROPE_PLAIN = 0,
    SZ_ROPE_LINEAR = 1,
    SZ_ROPE_BASE = 2,
    SZ_ROPE_RAMP = 3,
    SZ_ROPE_BANDS = 4
} sz_rope_stretch;

/* Host-only: rotary_dim / 2 angles per position, in radians, to
 * inv_freq[], and the magnitude (1 except RAMP).  rotary_dim even, base >
 * 1, factor >= 1 (all but PLAIN), original_len >= 1 and fast > slow > 0
 * (RAMP and BANDS); SZ_ERR_INVALID_ARGUMENT otherwise. */
sz_status sz_rope_frequencies(uint32_t rotary_dim, double base, int stretch, double factor,
                              double original_len, double slow, double fast, double *inv_freq,
                              float *magnitude);

/* Host-only: phases[i] = inv_freq[i] / (2 pi), its fraction in units of
 * 2^-64 turns, from n angles per position in radians (finite). */
sz_status sz_rope_phases(const double *inv_freq, uint64_t n, uint64_t *phases);

/* Norm and rotation of queries and keys in one pass: for every token and
 * head, y = x / sqrt(mean(x^2) + eps) * weight over the head's elements
 * (weight NULL: y = x), then the rotation of the token's position, in FP32,
 * rounded once to BF16.  (With a weight the squares are FP32 too: elements
 * of 2^60 and more in size, or with eps 0 heads all below 2^-60, give 0 or
 * infinities.)
 *   q, q_out / k, k_out  source (BF16 or F32) and BF16 destination, each
 *                        with n_tokens tokens; q or k (with its destination)
 *                        may be NULL
 *   d_q_weight, d_k_weight  optional device float[head_dim], 16-byte aligned
 *   d_positions          device i32[n_tokens], any values
 *   eps                  >= 0, finite (used with a weight)
 *   rope                 NULL or rotary_dim 0: norm only */
sz_status sz_qk_norm_rope(const sz_heads *q, const sz_heads *q_out, const float *d_q_weight,
                          const sz_heads *k, const sz_heads *k_out, const float *d_k_weight,
                          uint32_t head_dim, uint64_t n_tokens, const int32_t *d_positions,
                          float eps, const sz_rope *rope, hipStream_t stream);

/* Appends new tokens to the cache: token i of sequence s's n new ones goes
 * to cache position c = d_lens[s] - n + i, its keys normed (with a weight)
 * and rotated, its values as they are, both rounded to BF16; with q given,
 * its queries are normed and rotated to q_out in the same launch.  The
 * rotation's position is c, or d_positions[token] where given.  k and v
 * have cache->kv_heads heads; every other argument as in sz_qk_norm_rope.
 *   d_status  optional device i32[n_seqs]: SZ_OK, or
 *             SZ_ERR_INVALID_ARGUMENT for a sequence whose starts are out
 *             of range or order (an earlier start lies above its first row,
 *             a later one below its end), whose length is below its new tokens' count
 *             or past its pages, or one of whose written pages is NULL or
 *             misaligned.  Of such a sequence the tokens that have no place
 *             are not written and the others may be; nothing outside valid
 *             pages is touched. */
sz_status sz_kv_append(const sz_heads *k, const sz_heads *v, const float *d_k_weight,
                       const sz_heads *q, const sz_heads *q_out, const float *d_q_weight,
                       float eps, const sz_rope *rope, const int32_t *d_positions,
                       const sz_kv_cache *cache, const sz_batch *batch, int32_t *d_status,
                       hipStream_t stream);

/* Attention of every new token over its sequence's cache.  Token i of
 * sequence s's n new ones stands at position c = d_lens[s] - n + i; its
 * query head h attends to the keys of KV head h / (q heads / kv_heads):
 * those at j < d_lens[s], with `causal` j <= c, with window > 0 (causal
 * only) j > c - window.  Scores are scale * q.k, with softcap > 0 softcap *
 * tanh(scale * q.k / softcap).  A query that no key is visible to gives
 * zeros and a log-sum of -infinity.  A key or value that a query does not
 * see has no effect on it, whatever its bits.
 * Scores, the softmax's maximum and sum, and the accumulated output are
 * FP32; the weights are rounded to BF16 before they multiply the values,
 * whatever the output's type.  Weights are at most 2^8 and the sums are
 * divided at the end, so a row's scores must stay below 2^29 and the size of
 * its values times 2^8 times its keys below 2^127; beyond that its outputs
 * may be infinite, NaN or zero.  Scores that are all -infinity give what no
 * key gives.
 *   q         BF16, batch->n_tokens tokens, heads a multiple of kv_heads;
 *             n_tokens * heads < 2^31, and n_tokens * heads / 128 + 2 *
 *             n_seqs * kv_heads < 2^24
 *   out       BF16 or F32, as many heads
 *   d_lse     optional device float[n_tokens][q heads]: ln of the sum of
 *             exp(score) over the visible keys
 *   max_len   a host-side bound of d_lens (longer sequences are refused);
 *             0, or anything past it, means what the pages hold,
 *             pages_per_seq * page_tokens (2^30 at most).  Work is split for
 *             this bound, so it should not be far above the lengths.
 *   scale     > 0, softcap >= 0 (0: none); both, and scale / softcap, finite
 *             and below 1e38
 *   d_workspace, workspace_bytes   256-byte aligned, at least
 *             sz_attend_workspace_size(q->heads, cache, batch, max_len); any
 *             content; NULL where that is 0.  Calls (or replays of graphs)
 *             that may overlap need workspaces of their own.
 *   d_status  optional device i32[n_seqs]: SZ_OK, or
 *             SZ_ERR_INVALID_ARGUMENT for a sequence whose starts are out
 *             of range or order (an earlier start lies above its first row,
 *             a later one below its end), whose length is negative or above max_len,
 *             or one of whose pages with a visible token is NULL or
 *             misaligned.  The outputs of such a sequence are unspecified;
 *             nothing outside valid pages is read.
 * sz_attend_workspace_size reads n_seqs and n_tokens of the batch, not its
 * arrays; 0 also for invalid arguments.  Host-only. */
uint64_t sz_attend_workspace_size(uint64_t q_heads, const sz_kv_cache *cache,
                                  const sz_batch *batch, uint64_t max_len);
sz_status sz_attend_pages(const sz_heads *q, const sz_heads *out, float *d_lse,
                          const sz_kv_cache *cache, const sz_batch *batch, uint64_t max_len,
                          float scale, float softcap, int causal, uint64_t window,
                          void *d_workspace, uint64_t workspace_bytes, int32_t *d_status,
                          hipStream_t stream);

/* ---- a paged cache of latents ------------------------------------------
 * Latent attention keeps one row per token, whatever the heads: a latent of
 * latent_dim elements, from which every head's key and value are made, and
 * rotary_dim elements of the key that are rotated and shared by the heads.
 * The calls below append such rows and attend over them: in the absorbed
 * form, where the projection of a head's keys has been multiplied into its
 * query and the values' one is left to be applied to the output, so that a
 * row is key and value at once (single tokens, drafts), and in the expanded
 * form, where every head's keys and values have been made from the latents
 * (prompts).  Rules of the calls above apply: streams, graphs, overlaps,
 * row order, ragged batches, statuses. */
typedef struct {
    const void *const *d_pages; /* page c / page_tokens of sequence s: d_pages[s * table_pitch + ..] */
    uint64_t pages_per_seq;     /* as in sz_kv_cache */
    uint64_t table_pitch;
    uint64_t token_stride;      /* elements from a token's row to the next's in a page, at least */
                                /* latent_dim + rotary_dim; a multiple of 8, below 2^26 */
    uint32_t latent_dim;        /* a multiple of 8, 8 .. 512 */
    uint32_t rotary_dim;        /* a multiple of 8, 0 .. 64; its elements follow the latent's */
    uint32_t page_tokens;       /* a power of two, 16 .. 65536 */
} sz_latent_cache;

/* Appends new tokens' rows: latents normed over their latent_dim elements
 * (with a weight, as in sz_qk_norm_rope), rotary parts rotated, in FP32 and
 * rounded once to BF16; with q given, the rotary parts of the queries'
 * heads are rotated to q_out in the same launch.  Positions as in
 * sz_kv_append.
 *   latent    one head of latent_dim elements, BF16 or F32
 *   k_rotary  one head of rotary_dim elements; NULL where that is 0
 *   q, q_out  NULL, or rotary_dim > 0 and heads of as many elements: the
 *             queries' rotary parts and their BF16 destination (in place
 *             where q is BF16; usually the last elements of the rows that
 *             sz_attend_latent takes)
 *   d_weight  optional device float[latent_dim], 16-byte aligned
 *   rope      NULL or rotary_dim 0: no rotation; else of cache->rotary_dim
 *   d_status  as in sz_kv_append */
sz_status sz_latent_append(const sz_heads *latent, const float *d_weight, float eps,
                           const sz_heads *k_rotary, const sz_heads *q, const sz_heads *q_out,
                           const sz_rope *rope, const int32_t *d_positions,
                           const sz_latent_cache *cache, const sz_batch *batch,
                           int32_t *d_status, hipStream_t stream);

/* Attention of every new token over its sequence's latents, the absorbed
 * form: scores are scale * (query head . row), over latent_dim + rotary_dim
 * elements, the values a row's first latent_dim.  Positions, what a query
 * sees, empty queries, accuracy, max_len, workspace and statuses as in
 * sz_attend_pages, with one KV head, no window and no cap.
 *   q    BF16, heads of latent_dim + rotary_dim elements
 *   out  BF16 or F32, as many heads of latent_dim elements
 *   n_tokens * heads < 2^30, n_tokens * heads / 64 + 2 * n_seqs < 2^24 - 16 */
uint64_t sz_attend_latent_workspace_size(uint64_t heads, const sz_latent_cache *cache,
                                         const sz_batch *batch, uint64_t max_len);
sz_status sz_attend_latent(const sz_heads *q, const sz_heads *out, float *d_lse,
                           const sz_latent_cache *cache, const sz_batch *batch, uint64_t max_len,
                           float scale, int causal, void *d_workspace, uint64_t workspace_bytes,
                           int32_t *d_status, hipStream_t stream);

/* Attention of every new token over keys and values that have been expanded
 * from latents, every head with its own: sequence s has the rows
 * d_key_starts[s] .. + d_lens[s] - 1 of k, v and k_rotary.  Scores are scale *
 * (first key_dim elements of the query head . k + the following rotary_dim
 * ones . k_rotary); the rest as in sz_attend_latent.
 *   q         BF16, heads of key_dim + rotary_dim elements
 *   out       BF16 or F32, as many heads of value_dim elements
 *   k, v      BF16, as many heads of key_dim and value_dim elements, n_keys
 *             rows, token strides below 2^26; may be slices of one tensor
 *   k_rotary  BF16, one head (shared by all) or as many, of rotary_dim
 *             elements, n_keys rows; NULL where rotary_dim is 0
 *   key_dim, value_dim   multiples of 8, 8 .. 128
 *   rotary_dim           a multiple of 8, 0 .. 64
 *   d_key_starts  device i32[n_seqs]; any order, rows may be shared
 *   n_keys    < 2^31
 *   max_len   a host-side bound of d_lens (longer sequences are refused); 0, or
 *             anything past it, means n_keys.  The workspace's size goes by
 *             that bound; asked for with 0 it is enough for any
 *   n_tokens * heads < 2^31, n_tokens * heads / 128 + 2 * n_seqs * heads < 2^24
 *   d_status  SZ_ERR_INVALID_ARGUMENT also for a sequence whose rows do not
 *             lie in 0 .. n_keys */
uint64_t sz_attend_expanded_workspace_size(uint64_t heads, uint32_t value_dim,
                                           const sz_batch *batch, uint64_t max_len);
sz_status sz_attend_expanded(const sz_heads *q, const sz_heads *out, float *d_lse,
                             const sz_heads *k, const sz_heads *k_rotary, const sz_heads *v,
                             uint32_t key_dim, uint32_t rotary_dim, uint32_t value_dim,
                             const int32_t *d_key_starts, uint64_t n_keys,
                             const sz_batch *batch, uint64_t max_len, float scale, int causal,
                             void *d_workspace, uint64_t workspace_bytes, int32_t *d_status,
                             hipStream_t stream);

/* ---- eviction from a paged cache ---------------------------------------
 * A cache over its budget gives up the tokens that attention has looked at
 * the least: sz_weigh_pages adds up what each cached token has received,
 * step by step, beside sz_attend_pages; sz_evict_pages picks the tokens that
 * stay and copies their rows into other pages. */

/* The attention weight that cached tokens receive from a call's new tokens:
 * for KV head v of sequence s and every cached position j < d_lens[s]
 *   w[s][v][j] = keep * before[s][v][j] + sum exp(score - lse)
 * over the rows (new tokens and query heads of v) that see j, with the
 * scores and visibility of sz_attend_pages and the log-sums that it left in
 * d_lse.  The new tokens' own positions (the last ones) have no `before`; a
 * sequence without new tokens has keep * before.  Entries from d_lens[s] on are
 * left as they were.  A row whose log-sum is -infinity adds nothing; a row adds
 * nothing to keys that it does not see, whatever its bits and theirs.  FP32
 * throughout; the order of additions is fixed by the call's sizes and starts.
 * Only keys are read: d_v_pages of the cache may be the key table.
 *   q, d_lse   as sz_attend_pages took and left them (d_lse float[n_tokens]
 *              [q heads]); limits of q's heads and tokens as there
 *   d_before   optional device float[n_seqs][kv_heads][weights_pitch]; not read
 *              where it is NULL or keep is 0.  May be d_weights
 *   d_weights  device float[n_seqs][kv_heads][weights_pitch]
 *   weights_pitch  >= max_len (or what stands for it), < 2^31
 *   keep       finite
 *   max_len, scale, softcap, causal, window   as in sz_attend_pages
 *   d_workspace, workspace_bytes   256-byte aligned, at least
 *              sz_weigh_workspace_size of the same sizes; any content; NULL
 *              where that is 0
 *   d_status   as in sz_attend_pages; the weights of a sequence at fault are
 *              unspecified or as they were */
uint64_t sz_weigh_workspace_size(uint64_t q_heads, const sz_kv_cache *cache,
                                 const sz_batch *batch, uint64_t max_len);
sz_status sz_weigh_pages(const sz_heads *q, const float *d_lse, const float *d_before,
                         float *d_weights, uint64_t weights_pitch, float keep,
                         const sz_kv_cache *cache, const sz_batch *batch, uint64_t max_len,
                         float scale, float softcap, int causal, uint64_t window,
                         void *d_workspace, uint64_t workspace_bytes, int32_t *d_status,
                         hipStream_t stream);

/* Eviction: of each sequence's d_lens[s] cached tokens at most `budget`
 * stay: the first `first`, the last `recent`, and of those between them the
 * ones with the largest weights (of equal weights the earlier; NaN counts as
 * less than any number).  The rows of those that stay are copied, in
 * their order, to positions 0, 1, .. of the sequence's pages in `to`, their
 * weights to d_weights_to, and their old positions are written to d_kept (-1
 * from the number of those that stay on).  With weight_heads = kv_heads every
 * KV head keeps tokens of its own; with weight_heads = 1 all keep the same.
 * Keys stay as they were rotated: new tokens go on at the positions that they
 * would have had (d_positions of sz_kv_append).  All of a sequence that is
 * within the budget is copied as it is.
 *   d_weights     device float[n_seqs][weight_heads][weights_pitch]
 *   d_weights_to  device float[n_seqs][weight_heads][budget]; entries past
 *                 those that stay are left as they were
 *   d_kept        device i32[n_seqs][weight_heads][budget]
 *   from, to      caches of the same kv_heads and head_dim; pages and strides
 *                 may differ.  `to` must have room for min(budget, max_len)
 *                 tokens, and its written pages must not be pages that the
 *                 call reads: pages shared by other sequences stay as they are
 *   d_lens, d_lens_to   device i32[n_seqs], apart: tokens before and after
 *   n_seqs        0 .. 65535; n_seqs * weight_heads and n_seqs * budget / 16
 *                 below 2^22 and 2^24
 *   max_len       as in sz_attend_pages, <= weights_pitch
 *   budget        1 .. 2^30, >= first + recent
 *   d_status      optional device i32[n_seqs]: SZ_OK, or
 *                 SZ_ERR_INVALID_ARGUMENT for a sequence whose length is
 *                 negative or above max_len (none of its tokens stays), or one
 *                 of whose pages, up to its length in `from` and up to what
 *                 stays in `to`, is NULL or misaligned (rows there are not
 *                 copied) */
sz_status sz_evict_pages(const float *d_weights, uint64_t weight_heads, uint64_t weights_pitch,
                         const sz_kv_cache *from, const int32_t *d_lens, uint64_t n_seqs,
                         uint64_t max_len, uint64_t budget, uint64_t first, uint64_t recent,
                         const sz_kv_cache *to, float *d_weights_to, int32_t *d_kept,
                         int32_t *d_lens_to, int32_t *d_status, hipStream_t stream);

/* The same with the rows of d_weights_to weights_to_pitch floats apart (>=
 * budget, < 2^31) instead of budget: with a pitch that holds the tokens to
 * come, what stays is the next sz_weigh_pages' d_before as it is.  With
 * weight_heads = 1 that has kv_heads such rows a sequence: at kv_heads times
 * the distance what stays lies in the first, and the heads' sum goes on if the
 * others are zero.  Entries between the rows are left as they were. */
sz_status sz_evict_pages_pitched(const float *d_weights, uint64_t weight_heads,
                                 uint64_t weights_pitch, const sz_kv_cache *from,
                                 const int32_t *d_lens, uint64_t n_seqs, uint64_t max_len,
                                 uint64_t budget, uint64_t first, uint64_t recent,
                                 const sz_kv_cache *to, float *d_weights_to,
                                 uint64_t weights_to_pitch, int32_t *d_kept, int32_t *d_lens_to,
                                 int32_t *d_status, hipStream_t stream);

/* ---- compressed transfer to and from host memory ----------------------
 * The explainers present the codec as a way to shrink the KV transfer
 * between prefill and decode servers (introduction and "Les Resultats").
 * These calls wrap it around the transfer one GPU has, the PCIe copy to and
 * from host memory: the n words are cut into chunks of chunk_elems words
 * (the last one shorter), each chunk becomes an ordinary container with its
 * own codebook, and the codec runs on `stream` while earlier chunks'
 * containers are copied on a second stream, through three device staging
 * buffers.  Every call blocks the host until the transfer is complete.
 * Host buffers should be pinned (hipHostMalloc, or a PyTorch tensor with
 * pin_memory=True) for the copies to overlap.
 *
 * A transfer context (sz_ship_context_create) holds the copy stream, the
 * staging buffers and the events for one chunk size on the device current
 * when it is made; the _ctx calls use it and allocate nothing, except that
 * the first decode on a context enlarges its staging buffers to hold a
 * group of chunks (at least 2^24 words' worth, at most 128 MiB a buffer;
 * a decode moves small chunks a group at a time), and a decode with more
 * chunks than any before it grows the per-chunk status array.  A context
 * serves one transfer at a time.  The one-shot calls sz_ship_to_host /
 * sz_ship_from_host make a context, use it and release it.
 *
 * sz_ship_to_host: encode d_src[0..n) chunk by chunk into h_dst.
 *   chunk_elems  > 0, a multiple of 8 (keeps every chunk 16-byte aligned)
 *   h_dst        host buffer of h_capacity bytes; chunk c's container is at
 *                h_dst + h_offsets[c], h_offsets[c+1] - h_offsets[c] bytes
 *   h_offsets    host array of ceil(n / chunk_elems) + 1 entries, written
 * SZ_ERR_CAPACITY when the containers do not fit in h_capacity (found only
 * once a chunk's size is known: h_offsets is then valid up to the chunks
 * shipped before it).  SZ_ERR_INVALID_ARGUMENT for a bad chunk size, NULL
 * or misaligned pointers. */
sz_status sz_ship_to_host(const void *d_src, uint64_t n_elements, uint64_t chunk_elems,
                          void *h_dst, uint64_t h_capacity, uint64_t *h_offsets,
                          hipStream_t stream);

/* sz_ship_from_host: the reverse; h_src and h_offsets as sz_ship_to_host
 * wrote them, the words land in d_dst[0..n).  Returns SZ_ERR_CORRUPT (and
 * writes it to the optional device word *d_status, else SZ_OK there) when
 * an offset is out of order or a chunk's size cannot be a container of its
 * length (checked on the host before anything is copied), or when a chunk
 * fails a device-side check. */
sz_status sz_ship_from_host(const void *h_src, const uint64_t *h_offsets, uint64_t n_elements,
                            uint64_t chunk_elems, void *d_dst, int32_t *d_status,
                            hipStream_t stream);

/* A transfer context for chunks of chunk_elems words (> 0, a multiple of
 * 8) on the current device, to *ctx.  SZ_ERR_INVALID_ARGUMENT for a bad
 * chunk size or NULL ctx, SZ_ERR_HIP when an allocation fails (nothing is
 * then left allocated). */
typedef struct sz_ship_context sz_ship_context;
sz_status sz_ship_context_create(uint64_t chunk_elems, sz_ship_context **ctx);

/* Releases a context (NULL is ignored) after its copies have drained. */
void sz_ship_context_destroy(sz_ship_context *ctx);

/* sz_ship_to_host / sz_ship_from_host over a context, with its chunk size;
 * SZ_ERR_INVALID_ARGUMENT also when the context was made on another device. */
sz_status sz_ship_to_host_ctx(sz_ship_context *ctx, const void *d_src, uint64_t n_elements,
                              void *h_dst, uint64_t h_capacity, uint64_t *h_offsets,
                              hipStream_t stream);
sz_status sz_ship_from_host_ctx(sz_ship_context *ctx, const void *h_src,
                                const uint64_t *h_offsets, uint64_t n_elements, void *d_dst,
                                int32_t *d_status, hipStream_t stream);

/* Static English text for a status code (never NULL). */
const char *sz_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* SPLITZIP_H */
