/*
 * mrr.h -- libmrr: N-rank allreduce reduction for AMD MI355X (gfx950).
 *
 * One GPU holds the N "rank" buffers in its own HBM; each call performs every
 * rank's share of the reduction (or one chosen rank's share) in HIP kernels.
 *
 * Operations, and the passages that define them:
 *   - RS/AG zero-copy allreduce: "Support 2 ranks in AllreduceRsAgZeroCopy"
 *     (MSCCL++ PR #948), sections "why" and "what changed": rank r reduces
 *     chunk r of every rank's input and writes the result straight into every
 *     rank's output, with no scratch; it is compiled once per rank count,
 *     with the rank loops unrolled, for 2, 4, 8, 16 and 32 ranks; any other
 *     rank count is refused.
 *   - LL-packet allpair allreduce: MSCCL++ commit history (/src), entry fixing
 *     the allreduce_allpair_packet algorithm: packets go to a scratch area so
 *     the input is never overwritten, one workgroup sends, reduces and writes
 *     back, block/thread counts are validated, and the flag update works when
 *     a workgroup has fewer threads than flags.  Entry on the default flag
 *     buffer: one flag buffer shared by all algorithms so that switching
 *     between them by message size cannot hang.
 *   - FP8 E4M3B15 and accumulation precision: MSCCL++ commit history, entries
 *     adding the fp8_e4m3b15 datatype (4 exponent bits, 3 mantissa bits,
 *     bias 15, largest finite value 0.9375, converted through fp16) and the
 *     accumDtype parameter (AUTO resolves to the input type), and the entry
 *     adding ROCm support for the type with FP16/FP32 accumulation.
 *
 * Conventions shared by every entry point:
 *   - All data pointers are DEVICE pointers on the calling thread's current
 *     HIP device.  Pointer arrays (inputs[], outputs[], in_pkts[]) are HOST
 *     arrays of nranks device pointers; they are copied into the kernel
 *     arguments, so the host arrays may be reused as soon as the call returns.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *     Every call is stream-ordered and asynchronous: it validates its
 *     arguments on the host, launches, and returns without synchronising.
 *     No call allocates or frees memory, so calls may be captured in a HIP
 *     graph (the allocation-free entry point after its first call on a
 *     device, which sets up its workspace).
 *   - The caller owns every buffer.  Apart from the workspace of the
 *     allocation-free packet entry point (mrr_allreduce_packet_noalloc,
 *     below), the library keeps no device state; it caches only per-device
 *     properties (CU count, LDS size, occupancy).
 *   - Validation happens before any launch: on an error nothing is launched
 *     and the specific status is returned.  MRR_LOG=1 in the environment
 *     prints one stderr line per refused call (see mrr_reload_env).
 *   - count == 0 (or n == 0) returns MRR_OK without launching.
 *   - Element types travel as raw bits: f16 / bf16 as 16-bit IEEE binary16 /
 *     bfloat16, FP8 E4M3B15 as one byte (sign, 4-bit exponent with bias 15,
 *     3-bit mantissa; exponent 15 encodes inf (mantissa 0) and NaN).
 *   - Rounding is IEEE round-to-nearest-even everywhere.  f16 / bf16 overflow
 *     gives +-inf; FP8 E4M3B15 saturates to +-0.9375 and OCP FP8 E4M3FN to
 *     +-448 (also from +-inf); NaN gives NaN (FP8: 0x7F with the input's
 *     sign).  Denormals are kept.
 *   - OCP FP8 E4M3FN (MRR_FP8_E4M3FN) is accepted wherever FP8 E4M3B15 is as
 *     an input / accumulator / output type of the allreduce entry points
 *     (the pages' benchmarks reduce fp8_e4m3fn data; PR #948, "why").
 */
#ifndef MRR_H
#define MRR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mrr_status {
  MRR_OK = 0,
  MRR_EINVAL = 1,       /* bad argument: null pointer, rank or geometry out of range */
  MRR_EUNSUPPORTED = 2, /* rank count or type combination not provided */
  MRR_EALIGN = 3,       /* a pointer not aligned as the entry point requires */
  MRR_EOVERLAP = 4,     /* an output overlaps another buffer other than its own input */
  MRR_ESCRATCH = 5,     /* scratch or workspace smaller than its _bytes() function says */
  MRR_ETIMEDOUT = 6,    /* (device error word only) a packet poll exceeded max_spins */
  MRR_EHIP = 7          /* the HIP runtime refused the launch */
} mrr_status;

typedef enum mrr_dtype {
  MRR_AUTO = 0, /* accumulation: the input type; output: the input type */
  MRR_F32 = 1,
  MRR_F16 = 2,
  MRR_BF16 = 3,
  MRR_FP8_E4M3B15 = 4,
  MRR_FP8_E4M3FN = 5 /* OCP FP8 E4M3FN: bias 7, largest finite 448, 0x7F/0xFF NaN, no inf */
} mrr_dtype;

/* Packet / RS-AG crossover for mrr_allreduce, measured on one MI355X: 0.
 * There RS/AG is faster at every size (8 ranks of f16, per call under HIP
 * graph replay: 1.9 us against 5.7-8.8 us for allpair packets at 16-64 KiB
 * per rank, 3.6 us against 47.3 us at 1 MiB), because within one GPU it
 * needs no cross-rank synchronisation while packets double the bytes moved.
 * The pages' selectors, spanning GPUs, switch to RS/AG above 512 KiB
 * (Python default) or 2 MiB (NCCL shim). */
#define MRR_PACKET_MAX_BYTES_ONE_GPU 0

/* Largest rank count any entry point accepts. */
#define MRR_MAX_RANKS 32
/* Flag slots per rank in a packet flag buffer. */
#define MRR_PKT_FLAG_SLOTS 1024

/* --------------------------------------------------------------------------
 * RS/AG zero-copy allreduce ("Support 2 ranks in AllreduceRsAgZeroCopy",
 * sections "why" and "what changed").
 *
 * For every k < nranks and i < count:
 *   outputs[k][i] = round_out( x_0[i] + x_1[i] + ... + x_{nranks-1}[i] )
 * summed in rank order 0..nranks-1 starting from x_0 (so -0 sums stay -0).
 * The index space is split into nranks chunks of
 *   C = roundup(ceil(count / nranks), 256 / sizeof(input element))
 * elements (the last chunks may be short or empty); chunk r is rank r's
 * reduce-scatter share, and its reduced values are written to all nranks
 * outputs (the all-gather).  The result does not depend on the partition;
 * the 256-byte rounding keeps every chunk on the cache-line grid.
 *
 * mrr_allreduce_rsag: input type == output type == dtype (F32, F16, BF16 or
 *   FP8_E4M3B15), FP32 accumulation, every chunk.
 * mrr_allreduce_rsag_ex:
 *   in     F32 | F16 | BF16 | FP8_E4M3B15
 *   accum  AUTO (= in) | F32 | F16 (F16 and FP8 inputs) | BF16 (BF16 inputs) |
 *          FP8_E4M3B15 (FP8 inputs).  With a non-F32 accumulator every
 *          partial sum is rounded to that type.
 *   out    AUTO (= in); FP8 inputs may also produce F16 or F32.
 *   rank   -1: all chunks (every rank's share); 0..nranks-1: chunk `rank`
 *          only, i.e. one GPU's share at its real shape (reads count/nranks
 *          elements of every input, writes them to every output).
 *
 * Buffers: inputs[r] holds count input elements, outputs[k] room for count
 * output elements.  outputs[k] may be exactly inputs[k] (in place; only when
 * the input and output types have the same size); any other overlap between
 * an output and any buffer gives MRR_EOVERLAP.  Inputs may overlap each
 * other.  Pointers must be aligned to their element size (MRR_EALIGN);
 * 16-byte alignment of every pointer selects the vector kernels, otherwise a
 * slower element-wise kernel runs.
 * Errors: MRR_EUNSUPPORTED for nranks not in {2,4,8,16,32} or a type
 * combination not listed; MRR_EINVAL for null arrays/pointers or a rank
 * outside [-1, nranks); MRR_EHIP when the launch fails.
 * ------------------------------------------------------------------------ */
mrr_status mrr_allreduce_rsag(const void* const* inputs, void* const* outputs, size_t count,
                              mrr_dtype dtype, int nranks, void* stream);

mrr_status mrr_allreduce_rsag_ex(const void* const* inputs, void* const* outputs, size_t count,
                                 mrr_dtype in, mrr_dtype accum, mrr_dtype out, int nranks,
                                 int rank, void* stream);

/* --------------------------------------------------------------------------
 * RS/AG allreduce of FP8 inputs with two outputs from one pass ("MSCCL++
 * commit history for /src", FP8 accumulation entry: FP8 data reduced with
 * higher-precision accumulation; the FP8 workloads emit an f16 result and an
 * FP8 re-encode of the same sums).
 *
 * Same sum, partition and rank semantics as mrr_allreduce_rsag_ex with
 * in = FP8_E4M3B15 or FP8_E4M3FN; every reduced value is written twice:
 *   outputs[k][i]  = round_f16(sum)           (count f16 elements)
 *   outputs2[k][i] = round_in(sum)            (count codes of the input type,
 *                                              RNE, saturating as in the
 *                                              conversions above)
 * both rounded once from the accumulator (so outputs2 is not a rounding of
 * outputs).  Equivalent to two mrr_allreduce_rsag_ex calls (out = F16, then
 * out = in) but the inputs are read once: N*count*(1 + 2 + 1) bytes moved
 * instead of N*count*(1 + 2) + N*count*(1 + 1).
 *   accum  AUTO (= in) | F32 | F16
 * Buffers: every inputs[r], outputs[k] and outputs2[k] 16-byte aligned
 * (MRR_EALIGN otherwise); outputs2[k] may be exactly inputs[k]; any other
 * overlap of an output gives MRR_EOVERLAP.
 * Errors: MRR_EUNSUPPORTED for nranks not in {2,4,8,16,32} or another type;
 * MRR_EINVAL for null arrays/pointers or rank outside [-1, nranks);
 * MRR_EHIP when the launch fails.
 * ------------------------------------------------------------------------ */
mrr_status mrr_allreduce_rsag_dual(const void* const* inputs, void* const* outputs,
                                   void* const* outputs2, size_t count, mrr_dtype in,
                                   mrr_dtype accum, int nranks, int rank, void* stream);

/* --------------------------------------------------------------------------
 * LL-packet allpair allreduce (commit history: allreduce_allpair_packet fix;
 * default flag buffer entry).
 *
 * A packet is 8 bytes: payload word k of a rank's buffer (bytes [4k, 4k+4),
 * little-endian, bytes past the end read as zero) in the low 32 bits and a
 * 32-bit flag in the high 32 bits.  npkt = ceil(count * elem_size / 4).
 *
 * Each call takes F = (flag slot value) + 1, skipping 0 on 32-bit wrap.
 * Workgroup (rank d, block b) packs slice b of inputs[d] and stores the
 * packets into scratch[p][d][*] for every peer p != d (64-bit agent-scope
 * stores); it then polls scratch[d][s][*] of slice b for every s != d until
 * every packet carries F (wavefront-level vote, 64-bit agent-scope loads),
 * sums in rank order 0..nranks-1 -- taking its own contribution straight
 * from inputs[d] -- and writes slice b of outputs[d]; finally it sets every
 * flag slot j of rank d with j % B == b to F.  The inputs are never written.
 *
 * scratch:  device, 8-byte aligned, layout [dst][src][npkt] of uint64 packets,
 *           at least mrr_packet_scratch_bytes() bytes (else MRR_ESCRATCH);
 *           the self slots [d][d] are unused.  Zero it once before first use.
 * flags:    device, nranks * MRR_PKT_FLAG_SLOTS uint32, zero-filled once
 *           before first use (and whenever it is recycled).  Every call leaves
 *           every slot equal to the F it used, so count, geometry and the
 *           algorithm may change between calls without a hang, and graph
 *           replays advance F on the device.  All ranks' slots must hold the
 *           same value.  May be shared with later calls of any packet entry.
 *           Flag wrap: after 2^32 - 1 calls on one flag buffer F returns to
 *           1.  Scratch packets that an earlier, larger call wrote and no
 *           later call rewrote keep their old flags, which the wrapped
 *           sequence reaches again, and a poll could then take such a stale
 *           packet for a new one.  Re-zero the flags and the scratch together
 *           before 2^32 - 1 calls (about 2.4 hours of back-to-back 2 us
 *           calls).
 * inputs / outputs: device, 4-byte aligned (MRR_EALIGN), outputs[k] may be
 *           inputs[k] exactly; other overlaps give MRR_EOVERLAP.
 * dtype:    F32 | F16 | BF16 | FP8_E4M3B15 (output type == input type).
 * accum:    AUTO (= dtype) | F32 | F16 (F16 and FP8 data).
 * max_spins: bound on poll iterations per wavefront; on expiry the kernel
 *           writes MRR_ETIMEDOUT into *dev_err (if dev_err is not NULL; first
 *           error wins) and finishes; outputs are then undefined.  0 = no
 *           bound.  Read *dev_err after synchronising the stream.
 * blocks_per_rank / threads (_ex only): B and the workgroup size; 0 = auto.
 *           B must be in [1, MRR_PKT_FLAG_SLOTS]; threads a multiple of 64 in
 *           [64, 512]; nranks * B workgroups must fit on the GPU at once
 *           (every workgroup waits for its peers), else MRR_EINVAL.
 * Calls that overlap in time on the same scratch or flags race; calls on one
 * stream never overlap.
 * Co-residency is checked against an idle GPU.  Work running at the same time
 * on other streams (an RS/AG call, whose workgroups also hold LDS, or any
 * other kernel) only delays the packet workgroups that do not fit until it
 * drains.  But two packet calls running at the same time on different
 * streams can each hold workgroups that wait for peers the other keeps off
 * the GPU: order such calls on one stream, or give them a max_spins bound,
 * or set MRR_COOPERATIVE=1 (see mrr_reload_env) to have such launches
 * refused instead.
 * ------------------------------------------------------------------------ */
/* Scratch and flag sizes for the calls above; 0 for an unknown type, nranks
 * outside [1, 32], or a count the entry points refuse as too large. */
size_t mrr_packet_scratch_bytes(size_t count, mrr_dtype dtype, int nranks);
size_t mrr_packet_flag_bytes(int nranks);

mrr_status mrr_allreduce_packet(const void* const* inputs, void* const* outputs, void* scratch,
                                size_t scratch_bytes, uint32_t* flags, size_t count,
                                mrr_dtype dtype, mrr_dtype accum, int nranks,
                                uint32_t max_spins, uint32_t* dev_err, void* stream);

mrr_status mrr_allreduce_packet_ex(const void* const* inputs, void* const* outputs, void* scratch,
                                   size_t scratch_bytes, uint32_t* flags, size_t count,
                                   mrr_dtype dtype, mrr_dtype accum, int nranks,
                                   uint32_t max_spins, uint32_t* dev_err, int blocks_per_rank,
                                   int threads, void* stream);

/* --------------------------------------------------------------------------
 * LL-packet allpair allreduce that allocates nothing, for callers that cannot
 * allocate device memory or pass a workspace: code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc.
 *
 * Same operation, results and flag protocol as mrr_allreduce_packet, but the
 * scratch and the flag slots live in a workspace the library owns: one
 * statically sized device array per GPU, MRR_NOALLOC_SCRATCH_BYTES of packet
 * scratch plus the flag slots of 32 ranks (about 32.1 MiB in all), held on
 * every GPU the library runs on until the process ends.  The call allocates
 * and frees nothing.
 *   - A call needs nranks^2 * ceil(count * elem_size / 4) * 8 bytes of packet
 *     scratch (mrr_packet_scratch_bytes); above MRR_NOALLOC_SCRATCH_BYTES it
 *     returns MRR_ESCRATCH and launches nothing.  For example 8 ranks take up
 *     to 256 KiB per rank of f16, 32 ranks up to 16 KiB.
 *   - The first call on each device clears the workspace with a kernel on
 *     `stream`, ahead of its own kernel; it must not be made under stream
 *     capture (MRR_EINVAL, nothing set up).  Later calls may be captured.
 *   - Every call on one GPU shares that GPU's workspace, which keeps the last
 *     call's packets and flags; calls of any rank count, size and type
 *     continue one flag sequence.  Calls that overlap in time on one GPU
 *     (different streams without ordering, or concurrent graphs) race and may
 *     hang until max_spins: order them on one stream.
 *   - The flag sequence wraps after 2^32 - 1 calls; past that a stale packet
 *     could be taken for a new one (see the flag notes above), so a process
 *     making that many calls should use mrr_allreduce_packet with its own
 *     buffers, which it can re-zero.
 * inputs / outputs / dtype / accum / nranks / max_spins / dev_err as for
 * mrr_allreduce_packet; geometry is chosen automatically.
 * ------------------------------------------------------------------------ */
#define MRR_NOALLOC_SCRATCH_BYTES (32u << 20)

mrr_status mrr_allreduce_packet_noalloc(const void* const* inputs, void* const* outputs,
                                        size_t count, mrr_dtype dtype, mrr_dtype accum,
                                        int nranks, uint32_t max_spins, uint32_t* dev_err,
                                        void* stream);

/* --------------------------------------------------------------------------
 * Two-phase packet allreduce: reduce-scatter then all-gather, both in LL
 * packets (the "packet" allreduce the commit log lists beside allpair, in
 * the entry adding accumDtype; its structure is not on the pages, so this is
 * the RS/AG partition carried by packets).  The index space is split as for
 * RS/AG: chunk c = elements [c*C, (c+1)*C), C = roundup(ceil(count/N),
 * 16/elem_size), i.e. cw = C*elem_size/4 payload words per chunk.
 *   1. rank d sends chunk c of its input to rank c: rs[c][d][k] (c != d);
 *   2. rank c waits for rs[c][s] (s != c), sums chunk c in rank order with
 *      its own chunk read from its input, writes it to outputs[c] and sends
 *      it to every peer: ag[p][c][k] (p != c);
 *   3. rank p waits for ag[p][s] (s != p) and writes chunk s of outputs[p].
 * Every packet carries the call's flag F (same flag contract, flag buffer
 * and time-out behaviour as mrr_allreduce_packet; one flag buffer may serve
 * both packet entry points).  Per rank it moves about 10*S bytes against
 * (3 + 4(N-1))*S for allpair.
 * scratch: 8-byte aligned, mrr_packet_rsag_scratch_bytes() bytes: the rs
 *   region then the ag region, each [dst][src][cw] uint64 packets.  Zero it
 *   once before first use.
 * Other arguments and errors as mrr_allreduce_packet_ex.
 * ------------------------------------------------------------------------ */
/* 0 for an unknown type, nranks outside [1, 32], or a count refused as too large. */
size_t mrr_packet_rsag_scratch_bytes(size_t count, mrr_dtype dtype, int nranks);

mrr_status mrr_allreduce_packet_rsag(const void* const* inputs, void* const* outputs,
                                     void* scratch, size_t scratch_bytes, uint32_t* flags,
                                     size_t count, mrr_dtype dtype, mrr_dtype accum, int nranks,
                                     uint32_t max_spins, uint32_t* dev_err, int blocks_per_rank,
                                     int threads, void* stream);

/* --------------------------------------------------------------------------
 * Full-mesh allreduce (commit history: the entries adding accumDtype and
 * ROCm FP8 E4M3B15 support name a "fullmesh" allreduce beside the allpair
 * packet one; its steps are not on the pages, so this is the plain reading of
 * the name: every rank talks to every peer directly, by writes only, in plain
 * data rather than LL packets, each delivery signalled by a flag written
 * after it).  Chunks as the two-phase packet allreduce: C = roundup(ceil(count
 * / N), 16 / elem_size) elements, chunk c = elements [c*C, min((c+1)*C,
 * count)).  Workgroup (rank d, block b) takes slice b of every chunk:
 *   1. it writes slice b of chunk c of inputs[d] into inbox [c][d] of the
 *      scratch, for every peer c != d;
 *   2. it sets semaphore [c][d][b] = (uint64)F << 32 for every peer c != d
 *      (agent-scope release after the data);
 *   3. it waits until semaphore [d][s][b] carries F for every peer s
 *      (agent-scope acquire; bounded by max_spins), sums slice b of chunk d
 *      in rank order 0..nranks-1 -- its own part from inputs[d], the others
 *      from inbox [d][s] -- and writes it to chunk d of every outputs[k];
 *   4. it sets the flag slots j of rank d with j % B == b to F.
 * Per call it moves about (4N - 2) * S bytes (S = count * elem_size), against
 * 2N * S for RS/AG.
 * scratch: device, 16-byte aligned, mrr_fullmesh_scratch_bytes() bytes: the
 *   semaphores, N * N * MRR_PKT_FLAG_SLOTS uint64 [dst][src][slot], then the
 *   inboxes, N * N * C * elem_size bytes [dst][src][chunk].  Zero it once
 *   before first use (a semaphore must never hold a flag the sequence has
 *   not reached).  It may be shared with the packet entry points and the same
 *   flag buffer.
 * inputs / outputs: 16-byte aligned (MRR_EALIGN); outputs[k] may be
 *   inputs[k] exactly.  flags, dtype, accum, max_spins, dev_err,
 *   blocks_per_rank, threads and errors as mrr_allreduce_packet_ex (the
 *   auto geometry covers one 16-byte vector per lane per chunk).
 * ------------------------------------------------------------------------ */
size_t mrr_fullmesh_scratch_bytes(size_t count, mrr_dtype dtype, int nranks);

mrr_status mrr_allreduce_fullmesh(const void* const* inputs, void* const* outputs, void* scratch,
                                  size_t scratch_bytes, uint32_t* flags, size_t count,
                                  mrr_dtype dtype, mrr_dtype accum, int nranks,
                                  uint32_t max_spins, uint32_t* dev_err, int blocks_per_rank,
                                  int threads, void* stream);

/* --------------------------------------------------------------------------
 * One-call allreduce with algorithm selection ("Support 2 ranks in
 * AllreduceRsAgZeroCopy", section "why": selectors pick RS/AG zero-copy above
 * a message size and packets below it; section "what changed": rank counts
 * the RS/AG kernel does not cover could fall back to another algorithm).
 *
 * out type == dtype; accum as for the packet path (AUTO = dtype).
 *   - nranks in {2,4,8,16,32}, scratch and flags non-NULL, scratch_bytes >=
 *     mrr_packet_scratch_bytes(), count * elem_size <= packet_max_bytes and
 *     the (dtype, accum) pair has a packet kernel: the LL-packet allpair
 *     (same contract as mrr_allreduce_packet).
 *   - otherwise RS/AG over all chunks; a rank count in [1, 32] without a
 *     compiled kernel (1, 3, 5, 6, 7, 9, ...) runs the runtime-N RS/AG kernel,
 *     with the same results (sum in rank order 0..N-1).
 * MRR_PACKET_MAX_BYTES_ONE_GPU is the crossover measured on one MI355X (see
 * its definition); callers sharing work over several GPUs pick their own.
 * Errors as for the chosen path; nranks outside [1, 32] -> MRR_EUNSUPPORTED.
 * ------------------------------------------------------------------------ */
mrr_status mrr_allreduce(const void* const* inputs, void* const* outputs, size_t count,
                         mrr_dtype dtype, mrr_dtype accum, int nranks, void* scratch,
                         size_t scratch_bytes, uint32_t* flags, size_t packet_max_bytes,
                         uint32_t max_spins, uint32_t* dev_err, void* stream);

/* Receive step alone: for every k < npkts, wait until in_pkts[s][k] carries
 * flag_in for every s, sum the payload elements (4 / elem_size per word) in
 * rank order with accumulator accum, round to dtype and store
 * out_pkts[k] = (flag_out << 32) | word with a 64-bit agent-scope store.
 * in_pkts: host array of nranks device pointers (8-byte aligned); out_pkts
 * must not overlap them.  max_spins / dev_err as above.  No co-residency is
 * needed (the producers are outside the call), so any npkts works. */
mrr_status mrr_packet_reduce(const uint64_t* const* in_pkts, uint64_t* out_pkts, size_t npkts,
                             mrr_dtype dtype, mrr_dtype accum, int nranks, uint32_t flag_in,
                             uint32_t flag_out, uint32_t max_spins, uint32_t* dev_err,
                             void* stream);

/* pkts[k] = (flag << 32) | word_k(src) for k < ceil(nbytes / 4) (64-bit
 * agent-scope stores).  src: 4-byte aligned device buffer of nbytes bytes;
 * pkts: 8-byte aligned. */
mrr_status mrr_pack(const void* src, uint64_t* pkts, size_t nbytes, uint32_t flag, void* stream);
/* Writes the nbytes payload bytes of pkts into dst (4-byte aligned). */
mrr_status mrr_unpack(const uint64_t* pkts, void* dst, size_t nbytes, void* stream);

/* --------------------------------------------------------------------------
 * FP8 E4M3B15 codec (commit history: fp8_e4m3b15 datatype entry).
 * Decode is exact; encode rounds once, to nearest-even, saturating at
 * +-0.9375.  n elements; pointers aligned to their element size (MRR_EALIGN),
 * 16-byte alignment selects the vector kernels.  In and out must not overlap
 * (MRR_EOVERLAP).
 * ------------------------------------------------------------------------ */
mrr_status mrr_fp8b15_to_f16(const uint8_t* in, uint16_t* out, size_t n, void* stream);
mrr_status mrr_fp8b15_to_f32(const uint8_t* in, float* out, size_t n, void* stream);
mrr_status mrr_f16_to_fp8b15(const uint16_t* in, uint8_t* out, size_t n, void* stream);
mrr_status mrr_f32_to_fp8b15(const float* in, uint8_t* out, size_t n, void* stream);

/* --------------------------------------------------------------------------
 * Layer norm of a rank sum: what consumes the N partial results of a
 * row-parallel product, with the residual of the layer.
 *
 *   h[i][c]  = round_dtype( x_0 + x_1 + ... + x_{nranks-1} + residual )
 *   y[i][c]  = round_dtype( (h - mean_i) * rstd_i * weight[c] + bias[c] )
 *   mean_i = mean over c of h[i][c]; rstd_i = 1 / sqrt(var_i + eps), var_i the
 *   mean of (h - mean_i)^2 (biased)
 * summed in rank order in f32, the residual last; statistics in f32, of the
 * rounded h.
 *
 * inputs:    host array of nranks (1..32) device pointers to rows x cols
 *            elements of dtype (F32 | F16 | BF16), rows ld_in elements apart;
 *            they may overlap each other.
 * residual:  as an input; NULL = none.
 * weight, bias: cols elements of wdtype: F32, or the data type (AUTO);
 *            NULL = 1 and 0.
 * sum:       receives h, rows ld_out elements apart; NULL = not stored.
 * out:       receives y, rows ld_out elements apart.
 * mean, rstd: receive rows f32 values each; NULL = not stored.
 * sum and out may each be exactly one of the inputs or the residual, when
 * ld_in == ld_out; any other overlap of an output gives MRR_EOVERLAP.
 * Pointers are aligned to their element (MRR_EALIGN); no call is slower by
 * much for less than 16 bytes.
 * Errors: MRR_EUNSUPPORTED for another type or nranks outside [1, 32];
 * MRR_EINVAL for null pointers, cols 0 or over 2^20, ld_in or ld_out below
 * cols or over 2^31, rows over 2^31 or an eps that is negative or NaN.
 * rows == 0 launches nothing.
 * ------------------------------------------------------------------------ */
mrr_status mrr_layernorm_fwd(const void* const* inputs, int nranks, const void* residual,
                             const void* weight, const void* bias, void* sum, void* out,
                             float* mean, float* rstd, size_t rows, size_t cols, size_t ld_in,
                             size_t ld_out, float eps, mrr_dtype dtype, mrr_dtype wdtype,
                             void* stream);

/* --------------------------------------------------------------------------
 * Gradient of mrr_layernorm_fwd.  With xhat = (h - mean) * rstd and
 * g = dout * weight, mean() over a row:
 *   dsum    = round( rstd * (g - mean(g) - xhat * mean(g * xhat)) + dresidual )
 *   dweight = round( sum over rows of dout * xhat )
 *   dbias   = round( sum over rows of dout )
 * dsum is the gradient of every input and of the residual alike (each enters
 * the sum with factor 1).  Sums are f32 and taken in a fixed order: the same
 * call gives the same bits.
 *
 * dout, sum (the forward's h), dresidual (the gradient that h receives from
 * elsewhere, NULL = none): rows ld_in elements apart; dsum: rows ld_out apart.
 * mean, rstd: the forward's.  weight as in the forward; dweight, dbias: cols
 * elements of wdtype.  dsum, dweight and dbias may be NULL, not all three.
 * dsum may be exactly dout, sum or dresidual when ld_in == ld_out.
 * workspace: device, 16-byte aligned, mrr_layernorm_bwd_workspace_bytes(rows,
 * cols) bytes at least (else MRR_ESCRATCH), contents irrelevant before and
 * after; needed only with dweight or dbias.
 * rows == 0 sets dweight and dbias to zero.  Errors as in the forward.
 * ------------------------------------------------------------------------ */
size_t mrr_layernorm_bwd_workspace_bytes(size_t rows, size_t cols);

mrr_status mrr_layernorm_bwd(const void* dout, const void* sum, const void* weight,
                             const float* mean, const float* rstd, const void* dresidual,
                             void* dsum, void* dweight, void* dbias, size_t rows, size_t cols,
                             size_t ld_in, size_t ld_out, mrr_dtype dtype, mrr_dtype wdtype,
                             void* workspace, size_t workspace_bytes, void* stream);

/* --------------------------------------------------------------------------
 * Cross entropy of a linear layer whose vocabulary rows lie in nranks shards,
 * without the logits in memory.
 *
 *   z[t][v]  = sum over c of hidden[t][c] * weight[v][c]       (f32, not rounded)
 *   lse[t]   = log( sum over v of exp(z[t][v]) )
 *   loss[t]  = lse[t] - z[t][targets[t]]
 * v runs over the rows of shard 0, then of shard 1, and so on.
 *
 * hidden:  tokens x cols elements of dtype (F32 | F16 | BF16), rows ld_hidden
 *          elements apart.
 * weights: host array of nranks (1..32) device pointers; weights[r] is rows[r] x
 *          cols elements of dtype, rows ld_weight elements apart.  rows: host
 *          array; a shard may have no rows (its pointer is then not read).
 * targets: tokens 64-bit indices into the whole vocabulary.  ignore_index: the
 *          target of a token without a loss (its loss is 0, its lse is still
 *          computed); it may be any value.  Any other target outside [0, vocabulary)
 *          gives the loss NaN and counts as ignored in the gradient.
 * loss, lse: receive tokens f32 values each; one of them may be NULL.
 * The loss of a token that is sure of its target keeps its digits: it is the largest
 * logit less the target's, plus the log of a sum that is relative to the largest.
 * Every sum is f32.  f32 calls of few products (up to 4096 tokens; by time) multiply as
 * f32; others as sums of products of three bf16 parts, which hold an operand exactly (from
 * 2^-102 on).  What those leave out is 2^-26 of each product, less than an f32 product's
 * rounding, and no row's error depends on the size of another row.
 * workspace: device, 16-byte aligned, mrr_linear_xent_workspace_bytes(...,
 * backward 0) bytes at least (else MRR_ESCRATCH), contents irrelevant before and
 * after.  It may not overlap anything else.
 * Pointers are aligned to their element (MRR_EALIGN).  16-bit weights whose shards
 * are 16-byte aligned, with cols a multiple of 64 and ld_weight of 8 (and at most
 * 2^22), are read in place, and so are such hidden states in the forward; a forward of
 * up to 4 tokens or of few f32 products reads any operands in place.  Others are first
 * laid out in the workspace: hidden states whole, the vocabulary 256 MiB at a time (up
 * to 1 GiB where fewer rows would leave compute units idle, 256 rows at least).  Calls
 * whose weights (in the forward hidden states too) are read in place need only
 * mrr_linear_xent_workspace_bytes_in_place() bytes, which has no room for them; it
 * returns the other function's number for sizes that are never read in place.
 * The same call gives the same bits.  tokens == 0 launches nothing.
 * Errors: MRR_EUNSUPPORTED for another type or nranks outside [1, 32];
 * MRR_EINVAL for null pointers, cols 0 or over 2^20, tokens over 2^24, a
 * vocabulary of 0 or over 2^30 rows, or a row stride below cols or over 2^31;
 * MRR_EOVERLAP for an output that overlaps anything.
 * ------------------------------------------------------------------------ */
size_t mrr_linear_xent_workspace_bytes(size_t tokens, size_t cols, const size_t* rows, int nranks,
                                       mrr_dtype dtype, int backward);
size_t mrr_linear_xent_workspace_bytes_in_place(size_t tokens, size_t cols, const size_t* rows,
                                                int nranks, mrr_dtype dtype, int backward);

mrr_status mrr_linear_xent_fwd(const void* hidden, const void* const* weights, const size_t* rows,
                               int nranks, const int64_t* targets, int64_t ignore_index,
                               float* loss, float* lse, size_t tokens, size_t cols,
                               size_t ld_hidden, size_t ld_weight, mrr_dtype dtype,
                               void* workspace, size_t workspace_bytes, void* stream);

/* --------------------------------------------------------------------------
 * Gradient of mrr_linear_xent_fwd.
 *
 *   dz[t][v]       = (exp(z[t][v] - lse[t]) - [v == targets[t]]) * dloss[t]
 *   dhidden[t][c]  = round( sum over v of dz[t][v] * weight[v][c] )
 *   dweight[v][c]  = round( sum over t of dz[t][v] * hidden[t][c] )
 * The logits are computed again, a piece of the vocabulary at a time; the piece's
 * dz is held in dtype, up to 64 tokens in two parts (f32: in three bf16 parts, exactly);
 * sums are f32.  Of more than 64 tokens in 16 bits each dz is rounded once; what that takes
 * from a target's dz is given back to both gradients, so that only rows that are no token's
 * target show it (bf16: 0.0022 off in place of 0.0017, their own rounding).  f16: dz is scaled so that the largest |dloss| is 2^14, and is off by up to 2^-39
 * of the largest |dloss| as well: a token whose own is below 2^-20 of it loses digits.
 * Ignored tokens are left out: their dhidden is zero and nothing in their rows,
 * NaN included, reaches a gradient.
 *
 * hidden, weights, rows, targets, ignore_index: as in the forward.  lse: the
 * forward's.
 * dloss: gradient of token t's loss at dloss[t * dloss_stride]; stride 0 takes
 * one value for all (that of a mean or a sum).
 * dhidden: rows ld_hidden apart; NULL = not wanted.  It may be exactly hidden.
 * dweights: host array of nranks device pointers, rows ld_weight apart; NULL, or
 * an entry NULL = not wanted.  At least one output is wanted (else MRR_EINVAL).
 * workspace: as in the forward, with backward 1.
 * tokens == 0 sets the weight gradients to zero (no workspace needed).
 * Errors as in the forward, and MRR_EINVAL for a dloss_stride over 2^31.
 * ------------------------------------------------------------------------ */
mrr_status mrr_linear_xent_bwd(const void* hidden, const void* const* weights, const size_t* rows,
                               int nranks, const int64_t* targets, int64_t ignore_index,
                               const float* lse, const float* dloss, size_t dloss_stride,
                               void* dhidden, void* const* dweights, size_t tokens, size_t cols,
                               size_t ld_hidden, size_t ld_weight, mrr_dtype dtype,
                               void* workspace, size_t workspace_bytes, void* stream);

/* --------------------------------------------------------------------------
 * Head norms and rotation of a projection to queries, keys and values: what
 * consumes its N partial results before attention.
 *
 *   h    = round_dtype( x_0 + x_1 + ... + x_{nranks-1} )     summed in rank order in f32
 *   xhat = h / sqrt( mean over a head of h^2 + eps )
 *   y    = round_dtype( R( xhat * weight ) )      queries and keys, each with their weight
 *   y    = h                                      values
 * A row of the inputs holds heads[0] query heads, heads[1] key heads and heads[2] value
 * heads of head_dim elements, side by side.  R rotates the first rot_dim elements of a head
 * by the token's angles and leaves the others: a pair (a, b) becomes (a cos - b sin, b cos +
 * a sin).  pairs 0: element i < rot_dim / 2 pairs with i + rot_dim / 2; pairs 1: 2 i with
 * 2 i + 1.  All in f32, rounded once.  So are the squares: a head whose squares sum to more than
 * f32 holds (all elements over 1.8e19 / sqrt(head_dim)) becomes zeros, and its gradients with it;
 * without eps one of elements below 1e-18 loses digits, and one whose squares vanish (below
 * 1e-23) becomes infinite, zeros NaN.
 *
 * inputs:    host array of nranks (1..32) device pointers to rows of dtype (F32 | F16 |
 *            BF16), one a token, ld_in elements apart; they may overlap each other.
 * q_weight, k_weight: head_dim elements of wdtype: F32, or the data type (AUTO); NULL = 1.
 * table:     table_rows rows of rot_dim f32: rot_dim / 2 cosines, then their sines, of
 *            each position (NULL with rot_dim 0).
 * positions: 64-bit row of the table for each token; NULL = 0, 1, 2, ...  A token whose
 *            position is negative fills up a padded batch: nothing of it is read, and no
 *            output of it is written.  A position of table_rows or more rotates by NaN.
 * sum:       receives h (all heads), rows ld_in apart; NULL = not stored.
 * outs:      host array of three device pointers: y of the queries, keys and values, or
 *            NULL = not stored (as where there are no such heads).  Element d of head j of
 *            token t lies at t * ld_outs[k] + j * head_strides[k] + d (so token by token
 *            or head by head, in a buffer of its own or as columns of a wider one).
 * sum may be exactly one of the inputs, and each of outs exactly its heads' columns of one;
 * any other overlap of an output gives MRR_EOVERLAP.  Outputs of the same strides may lie
 * between each other (query, key and value of head 0, then of head 1).  Pointers are aligned to their
 * element (MRR_EALIGN).  The same call gives the same bits.  tokens == 0 launches nothing.
 * Errors: MRR_EUNSUPPORTED for another type or nranks outside [1, 32]; MRR_EINVAL for null
 * pointers, head_dim 0 or over 512, rot_dim odd or over head_dim, a head count over
 * 65535 or none at all, tokens over 2^31, ld_in below a row or over 2^31, a stride between
 * tokens over 2^31 or between heads over 2^40, strides that put two elements in one place or
 * keep neither tokens nor heads apart as rows, table_rows of 0 or over 2^31, without positions more
 * tokens than table_rows, and an eps that is negative or NaN.
 * ------------------------------------------------------------------------ */
mrr_status mrr_qknorm_rope_fwd(const void* const* inputs, int nranks, const void* q_weight,
                               const void* k_weight, const float* table, size_t table_rows,
                               const int64_t* positions, void* sum, void* const* outs,
                               size_t tokens, const size_t* heads, size_t head_dim,
                               size_t rot_dim, int pairs, size_t ld_in, const size_t* ld_outs,
                               const size_t* head_strides, float eps, mrr_dtype dtype,
                               mrr_dtype wdtype, void* stream);

/* --------------------------------------------------------------------------
 * Gradient of mrr_qknorm_rope_fwd.  With u = R^T(dout), g = u * weight and rs =
 * 1 / sqrt( mean(h^2) + eps ) of a head:
 *   dsum    = round( rs * (g - xhat * mean(g * xhat)) )      queries and keys
 *   dsum    = dout                                           values
 *   dweight = round( sum over tokens and their heads of u * xhat )
 * dsum is the gradient of every rank's input alike.  Sums are f32 and taken in a fixed order:
 * the same call gives the same bits.
 *
 * douts, ld_douts, head_strides: gradients of the forward's outs, laid out as those; NULL =
 * zero.  sum: the forward's h (with one rank its input), and dsum: rows ld_in apart.
 * dsum, dq_weight and dk_weight may be NULL, not all three.  Rows of dsum of tokens with a
 * negative position are zero, and nothing of them reaches a gradient.
 * dsum may be exactly sum.
 * workspace: device, 16-byte aligned, mrr_qknorm_rope_bwd_workspace_bytes(tokens, heads,
 * head_dim) bytes at least (else MRR_ESCRATCH), contents irrelevant before and after;
 * needed only with dq_weight or dk_weight.
 * tokens == 0 sets the weight gradients to zero.  Errors as in the forward.
 * ------------------------------------------------------------------------ */
size_t mrr_qknorm_rope_bwd_workspace_bytes(size_t tokens, const size_t* heads, size_t head_dim);

mrr_status mrr_qknorm_rope_bwd(const void* const* douts, const void* sum, const void* q_weight,
                               const void* k_weight, const float* table, size_t table_rows,
                               const int64_t* positions, void* dsum, void* dq_weight,
                               void* dk_weight, size_t tokens, const size_t* heads,
                               size_t head_dim, size_t rot_dim, int pairs, size_t ld_in,
                               const size_t* ld_douts, const size_t* head_strides, float eps,
                               mrr_dtype dtype, mrr_dtype wdtype, void* workspace,
                               size_t workspace_bytes, void* stream);

/* --------------------------------------------------------------------------
 * Matrices made orthogonal by Newton-Schulz products.
 *
 *   X_0 = in / ( |in| + eps )                       |.| the Frobenius norm of a matrix
 *   A = X X^T,  X <- a X + (b A + c A A) X          steps times
 *   out = round_dtype( X )
 * which takes each singular value s of X_0 through a s + b s^3 + c s^5 at each step and
 * leaves the singular vectors (of matrices with more rows than columns the transpose is
 * taken through the same steps).
 *
 * in, out: batch matrices of rows x cols elements of dtype (F32 | F16 | BF16), rows ld_in
 *          (ld_out) and matrices stride_in (stride_out) elements apart.
 * coefficients: host array of a, b, c of each step; NULL = 3.4445, -4.7750, 2.0315 at
 *          every step, which bring singular values from 0.01 of the norm up to within 0.68
 *          and 1.14 in 5 steps.
 * products: precision of the products.  F32 (AUTO): operands in two f16 parts (22 bits),
 *          three products of them for each: results as exact as f32 products give (5 steps:
 *          off by 1e-6 to 3e-6 of their norm for noise, and where one direction stands alone by
 *          5e-5 for 65 a side, 3e-4 for 4096).  F16, where speed counts for more: operands of 11 bits, diagonals and what
 *          a step adds to in f32 beside them.  Its results are off by some 1e-3 of their norm
 *          for noise; equal rows round alike and their errors add, up to 3e-2 for blocks of
 *          equal values (bf16 itself rounds by 1.7e-3).  Matrices with a side of 64 or
 *          less always take F32.
 * Norms and sums are f32 or f64.  A matrix of zeros gives zeros; one that holds NaN or an
 * infinity gives NaN.  The same call gives the same bits.
 * out may be exactly in, with the same strides; any other overlap gives MRR_EOVERLAP, as do
 * results of which neither the matrices nor their rows lie apart.
 * workspace: device, 16-byte aligned, mrr_orthogonalize_workspace_bytes(...) bytes at least
 * (else MRR_ESCRATCH), contents irrelevant before and after.
 * batch == 0 launches nothing.
 * Errors: MRR_EUNSUPPORTED for another type or precision; MRR_EINVAL for null pointers,
 * rows or cols of 0 or over 65536, a batch over 65535, steps outside [1, 64], a stride below
 * a row or over 2^31 (matrices: 2^40), an eps that is negative or not finite, and coefficients
 * with which singular values could come within 1 % of 7.5 before a step, or |b x + c x^2|
 * pass 1000 for any x up to their squares.
 * ------------------------------------------------------------------------ */
size_t mrr_orthogonalize_workspace_bytes(size_t rows, size_t cols, size_t batch, mrr_dtype dtype,
                                         mrr_dtype products);

mrr_status mrr_orthogonalize(const void* in, void* out, size_t rows, size_t cols, size_t ld_in,
                             size_t ld_out, size_t batch, size_t stride_in, size_t stride_out,
                             int steps, const float* coefficients, float eps, mrr_dtype dtype,
                             mrr_dtype products, void* workspace, size_t workspace_bytes,
                             void* stream);

/* --------------------------------------------------------------------------
 * The weights' update by mrr_orthogonalize (the Muon optimiser's step), from every rank's
 * gradients to every rank's weights.
 *
 *   g            = grad_scale * ( G_0 + G_1 + ... + G_{nranks-1} )      in rank order, f32
 *   momentum_out = mu * momentum + g
 *   u            = g + mu * momentum_out (nesterov), or momentum_out
 *   weights_out[r] = round_wdtype( (1 - decay) * weight - rate * X )    for every r,
 * X what mrr_orthogonalize makes of u in f32, not rounded before.  rate and decay are
 * taken as they are: factors for a matrix's sides, and rate * weight decay, are the caller's.
 *
 * grads:   host array of nranks (1..32) device pointers to batch matrices of gdtype (F32 |
 *          F16 | BF16), rows ld_grad, matrices stride_grad elements apart; they may overlap.
 * weight:  batch matrices of wdtype (F32 | F16 | BF16, or AUTO = gdtype), rows ld_weight,
 *          matrices stride_weight elements apart; weights_out: host array of nranks device
 *          pointers to such matrices.
 * momentum, momentum_out: f32, laid out as the weights; momentum NULL = zeros (a first step).
 * weights_out[r] may be exactly weight, and momentum_out exactly momentum; any other overlap
 * of an output gives MRR_EOVERLAP.
 * products: as in mrr_orthogonalize.
 * workspace: as there, mrr_muon_workspace_bytes(...) bytes at least, which takes wdtype AUTO too.
 * Factors are values of the call: a captured graph replays those it was captured with.
 * Errors as there; MRR_EUNSUPPORTED for nranks outside [1, 32]; MRR_EINVAL for a factor that
 * is not finite.
 * ------------------------------------------------------------------------ */
size_t mrr_muon_workspace_bytes(size_t rows, size_t cols, size_t batch, int nesterov,
                                mrr_dtype wdtype, mrr_dtype products);

mrr_status mrr_muon_step(const void* const* grads, int nranks, float grad_scale,
                         const float* momentum, float* momentum_out, float mu, int nesterov,
                         const void* weight, void* const* weights_out, float rate, float decay,
                         size_t rows, size_t cols, size_t ld_grad, size_t ld_weight, size_t batch,
                         size_t stride_grad, size_t stride_weight, int steps,
                         const float* coefficients, float eps, mrr_dtype gdtype, mrr_dtype wdtype,
                         mrr_dtype products, void* workspace, size_t workspace_bytes,
                         void* stream);

/* --------------------------------------------------------------------------
 * Copy-kernel calibration (measurement aid, not part of the reduction).
 * Copies nbytes from src to dst with the launch scheme of the RS/AG kernels
 * (one single-wave workgroup per tile, residency capped through an unused
 * LDS reservation, non-temporal 16-byte loads and stores): the same 1:1 mix
 * of streaming reads and writes as a reduction, without its arithmetic, so
 * its bandwidth is the practical ceiling a reduction is read against.
 * src and dst: device pointers, 16-byte aligned (MRR_EALIGN), ranges
 * disjoint (MRR_EOVERLAP); nbytes == 0 launches nothing; nbytes over 1 TiB
 * -> MRR_EINVAL.  Stream-ordered and asynchronous; allocates nothing.
 * ------------------------------------------------------------------------ */
mrr_status mrr_stream_copy(const void* src, void* dst, size_t nbytes, void* stream);

/* --------------------------------------------------------------------------
 * HBM placement of the simulated rank buffers (one GPU holds all N).
 *
 * When the N same-size rank buffers of one side (inputs, or outputs) are
 * carved from one device allocation, consecutive buffers should be
 * mrr_rank_buffer_pitch(bytes, nranks) bytes apart: bytes rounded up to
 * 4 KiB plus a stagger of 4 KiB (nranks < 16) or 3 KiB (nranks >= 16); from
 * 4 ranks up, when the rounded size is an odd multiple of 128 MiB, 5 KiB and
 * 8 KiB instead (8 x 128 MiB bf16: 0.74 -> 0.80 of the HBM peak).
 * Buffers spaced by a large power of two put the 2N equal-offset streams of
 * a reduction on the same DRAM channels; the stagger spreads them.  Measured
 * on MI355X with the RS/AG kernel, 8 x 64 MiB f16: 186.8 us with one
 * allocation per buffer, 180-181 us at this pitch, 205 us at an exact 64 MiB
 * pitch.  At 16 and 32 ranks (64 and 256 MiB each, mean of three runs) a
 * 3 KiB stagger gives 5.62 / 5.47 TB/s (N=16) and 5.28 / 5.10 TB/s (N=32),
 * against 5.31 / 5.55 and 5.17 / 5.13 at 2 KiB and 4.97-5.38 at 4 KiB.
 * Advisory only: every entry point accepts any placement.  Returns 0 for
 * bytes == 0 or nranks < 1.
 * ------------------------------------------------------------------------ */
size_t mrr_rank_buffer_pitch(size_t bytes_per_rank, int nranks);

/* --------------------------------------------------------------------------
 * Environment overrides (diagnostics and tuning; none changes a result).
 *   MRR_LOG=1          one stderr line per refused call
 *   MRR_MAX_GRID=<g>   at most g workgroups per RS/AG, codec or copy launch
 *                      (each then walks several tiles)
 *   MRR_LDS_CAP=0      persistent grids without the LDS reservation that caps
 *                      residency (frees the LDS for concurrent kernels)
 *   MRR_RSAG_WPC, MRR_RSAG_ANY_M, MRR_RSAG_SMALL=0, MRR_CODEC_U, MRR_CODEC_WPC
 *                      replace entries of the measured launch tables
 *   MRR_COOPERATIVE=1  launch the kernels whose workgroups wait for each other
 *                      (allpair, two-phase packets, full mesh) with
 *                      hipLaunchCooperativeKernel: a grid that cannot be
 *                      resident at once (for instance behind work on other
 *                      streams) is then refused at launch (MRR_EHIP) instead
 *                      of waiting; costs about 15 us per eager call on MI355X
 * They are read once, when the library is loaded.  mrr_reload_env() reads
 * them again (for tests and tuning sweeps that change them in-process); calls
 * running on other threads meanwhile see either the old or the new values.
 * ------------------------------------------------------------------------ */
void mrr_reload_env(void);

/* Static description of a status code (never NULL). */
const char* mrr_status_string(mrr_status status);

/* Library version, major * 10000 + minor * 100 + patch. */
int mrr_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MRR_H */
