/*
 * vr.h -- C ABI of the virtual-rank ring AllReduce library (libvr.so).
 *
 * N "virtual ranks" each own one send buffer and one receive buffer of `count`
 * elements, all on the same GPU. vrAllReduce leaves in every receive buffer
 * the elementwise reduction of the N send buffers, computed by the ring
 * schedule of NCCL's ring AllReduce: per channel, N-1 reduce-scatter stages
 * then N-1 all-gather stages, moving chunks from rank r to rank r+1 through
 * per-edge FIFO staging buffers in one of three protocol formats.
 *
 * The reduction order is fixed by the schedule ("NCCL 原始碼解讀：一個
 * AllReduce 的 GPU 旅程", ch.2 §2.3, RingARAlgorithm::getNextSendAddr): within
 * each loop of N*chunk elements of a channel, chunk c is first sent by rank
 * c+1 and accumulates ranks c+2, ..., c in ring order, op(incoming, own),
 * rounded to the element type after every op. Results are therefore bit-exact
 * reproducible for every dtype, including floating point, for a given
 * (nRanks, nChannels, chunkBytes, count).
 *
 * Conventions for every entry point:
 *  - Pointers named "device" must be device (or managed) memory of the GPU
 *    that was current when the communicator was created. Pointers named
 *    "host" are ordinary host memory read during the call only.
 *  - No call retains a caller pointer after it returns, except that device
 *    buffers passed to vrAllReduce are accessed by the enqueued kernel until
 *    it completes on `stream`.
 *  - A communicator is not thread-safe; calls on one communicator must be
 *    issued from one thread at a time and enqueued on one stream (the same
 *    stream for every vrAllReduce on that communicator), like an NCCL
 *    communicator ("NCCL 原始碼解讀", ch.2 §2.1).
 *  - Errors are returned, never raised; no entry point aborts the process.
 */
#ifndef VR_H_
#define VR_H_

#include <stddef.h>
#include <stdint.h>

/* Exported symbol marker: the library is built with hidden visibility and
 * exports exactly the entry points declared here. */
#if defined(__GNUC__)
#define VR_API __attribute__((visibility("default")))
#else
#define VR_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Opaque communicator handle (analog of ncclComm_t, "NCCL 原始碼解讀", ch.2
 * §2.1): owns the FIFO arena, the control words, the status word and the
 * per-call step base. Checked against a registry of live handles, so a
 * destroyed handle is rejected with vrInvalidArgument. */
typedef struct vrComm* vrComm_t;

/* Result codes. Mirror the shape of ncclResult_t ("NCCL 原始碼解讀", ch.1
 * §1.2 and ch.3 §3.1: invalid argument / invalid usage / internal error, and
 * ch.2 §2.1 asyncResult for errors found after enqueue). */
typedef enum {
  vrSuccess = 0,
  vrInvalidArgument = 1, /* null pointer, bad rank/channel count, unknown enum,
                            misaligned pointer, chunkBytes not a multiple of 16,
                            or a handle that is not a live communicator */
  vrInvalidUsage = 2,    /* valid arguments the device cannot run: too many
                            ranks x channels to be co-resident, FIFO too large */
  vrCudaError = 3,       /* a CUDA runtime call failed */
  vrInternalError = 4,   /* a bug in this library */
  vrTimeout = 5,         /* a device-side wait gave up (sticky, see below) */
  vrNumResults = 6
} vrResult_t;

/* FIFO protocols ("NCCL 原始碼解讀", ch.2 §2.4; bandwidth factors ch.5 §三):
 *  Simple: whole slots, one tail counter per slot step (producer) and one head
 *          counter (consumer), each on its own 128-byte line.
 *  LL:     16-byte lines of two 8-byte words {32-bit payload, 32-bit flag};
 *          data and flag arrive together, 50 % payload.
 *  LL128:  128-byte lines of 120 payload bytes and an 8-byte flag, 120/128
 *          payload. */
typedef enum { vrProtoSimple = 0, vrProtoLL = 1, vrProtoLL128 = 2, vrNumProtos = 3 } vrProto_t;

/* Element types. float16 is IEEE binary16, bfloat16 the upper half of binary32.
 * vrFloat8e4m3 and vrFloat8e5m2 are the OCP 8-bit floating-point formats
 * (E4M3: bias 7, no infinities, 0x7F/0xFF NaN, largest finite 448; E5M2:
 * bias 15, IEEE-like infinities and NaNs, largest finite 57344), the FP8
 * types that NCCL reduces on sm90 and later ("NCCL 原始碼解讀", ch.6, the FP8
 * type check). Their sum and product are computed exactly and rounded to
 * nearest even, a result past the largest finite value (or infinite)
 * saturating to it with its sign. */
typedef enum {
  vrInt8 = 0, vrUint8 = 1, vrInt32 = 2, vrUint32 = 3, vrInt64 = 4, vrUint64 = 5,
  vrFloat16 = 6, vrBfloat16 = 7, vrFloat32 = 8, vrFloat64 = 9, vrFloat8e4m3 = 10,
  vrFloat8e5m2 = 11, vrNumTypes = 12
} vrDataType_t;

/* Reductions. Integer sum and prod wrap (two's complement); max/min are
 * a > b ? a : b and a < b ? a : b (NaN behaviour unspecified).
 * vrAvg is the sum divided by nRanks, computed as the device op the host op
 * turns into ("NCCL 原始碼解讀", ch.6, hostToDevRedOp): for floating types
 * every rank's element is first multiplied by 1/nRanks (the factor rounded to
 * the element type, each product rounded to it), then summed in the ring's
 * order; for integer types the wrapped sum is divided by nRanks afterwards,
 * truncating toward zero (C division). Values >= vrNumOps are pre-multiplied
 * sums made by vrRedOpCreatePreMulSum on one communicator. */
typedef enum {
  vrSum = 0, vrProd = 1, vrMax = 2, vrMin = 3, vrAvg = 4, vrNumOps = 5
} vrRedOp_t;

/* Largest supported nRanks. */
#define VR_MAX_RANKS 128
/* Largest supported nChannels. */
#define VR_MAX_CHANNELS 128

/* Create a communicator for nRanks virtual ranks on the current CUDA device.
 * ("NCCL 原始碼解讀", ch.1 §1.2 ncclCommInitAll; ch.3 §3.3 commAlloc.)
 *  comm       [out, host] receives the handle; unchanged on error.
 *  nRanks     1 .. VR_MAX_RANKS.
 *  nChannels  1 .. VR_MAX_CHANNELS: the buffer is split into nChannels
 *             contiguous ranges (each divUp(count, nChannels) rounded up to 16
 *             bytes of elements), reduced independently and concurrently
 *             ("NCCL 原始碼解讀", ch.2 §2.2).
 *  proto      FIFO protocol.
 *  chunkBytes payload bytes per ring chunk; a multiple of 16, >= 16. It fixes
 *             the loop size N*chunkBytes and so the reduction order.
 * Allocates (cudaMalloc) the FIFO arena and control words, and a pinned host
 * status mirror; zeroes them. Environment knobs that never change results:
 * VR_FIFO_SLOT_BYTES (multiple of 256, 1 KiB..1 MiB), VR_FIFO_DEPTH
 * (2..64), VR_TRANSPORT (auto|global|warp|warpcluster), VR_CLUSTER_CTAS
 * (warpcluster: CTAs C a ring spans, 2 <= C <= min(16, nRanks) with
 * ceil(nRanks / C) <= 16), VR_FIFO_IN_DEPTH, VR_LATENCY_KERNEL (0: calls that
 * fit one pass of their rings, and Simple calls on rings inside one CTA, stay
 * on the general kernel), VR_TIMEOUT_MS,
 * VR_DEBUG (print the plan). Test only: VR_DEBUG_SILENT_RANK=k
 * makes virtual rank k never signal its neighbours, so that the others' waits
 * run out (vrTimeout). */
VR_API vrResult_t vrCommCreate(vrComm_t* comm, int nRanks, int nChannels, vrProto_t proto,
                        size_t chunkBytes);

/* Enqueue one AllReduce on `stream` (a cudaStream_t; NULL = legacy default).
 * ("NCCL 原始碼解讀", ch.1 §1.3 ncclAllReduce.)
 *  sendbufs [host array of nRanks device pointers] rank r's input; read only.
 *  recvbufs [host array of nRanks device pointers] rank r's output. In place
 *           (sendbufs[r] == recvbufs[r]) is allowed; other overlaps are not.
 *  count    elements per rank. 0 returns vrSuccess and launches nothing; the
 *           buffer pointers are then not examined (they may be NULL).
 *  dtype, op  element type and reduction.
 * Every pointer must be aligned to the element size; 16-byte-aligned buffers
 * take the vectorised path. The two host arrays are read during the call only.
 * Asynchronous: returns once the work is enqueued; synchronise `stream` before
 * reading the outputs. nRanks == 1 is a device-to-device copy (a scaling
 * kernel for a floating vrAvg or a pre-multiplied sum).
 * vrAvg and pre-multiplied sums run on the warp transports (vrCommGetInfo
 * transport 2 or 3) only: vrInvalidUsage on the others.
 * Returns vrTimeout without enqueuing if an earlier call on this communicator
 * timed out (sticky, like NCCL's asyncResult): destroy the communicator. */
VR_API vrResult_t vrAllReduce(vrComm_t comm, const void* const* sendbufs, void* const* recvbufs,
                       size_t count, vrDataType_t dtype, vrRedOp_t op, void* stream);

/* ReduceScatter on the ring: the reduce-scatter half of the AllReduce
 * schedule ("NCCL 原始碼解讀", ch.2 §2.3, the first (N-1)·chunkSteps steps
 * of nStepsPerLoop; traffic factor nRanks, ch.6 §五). Block b is folded
 * from rank b+1 around the ring to rank b, op(incoming, own), rounded to
 * the element type after every op.
 *  sendbufs [host array of nRanks device pointers] rank r's input of
 *           nRanks * recvcount elements; block b = elements
 *           [b * recvcount, (b + 1) * recvcount).
 *  recvbufs [host array of nRanks device pointers] rank r's output of
 *           recvcount elements: the reduction of block r. In place:
 *           recvbufs[r] == sendbufs[r] + r * recvcount elements.
 * Same rules as vrAllReduce otherwise. Runs on the warp transports
 * (vrCommGetInfo transport 2 or 3); vrInvalidUsage on the others. */
VR_API vrResult_t vrReduceScatter(vrComm_t comm, const void* const* sendbufs,
                                  void* const* recvbufs, size_t recvcount, vrDataType_t dtype,
                                  vrRedOp_t op, void* stream);

/* AllGather on the ring: the all-gather half of the schedule. Rank r's
 * output of nRanks * sendcount elements holds rank b's input in block b. The
 * data moves as bytes (as NCCL converts AllGather to int8, "NCCL 原始碼解讀",
 * ch.6); dtype only sets the element size.
 *  sendbufs [host array of nRanks device pointers] sendcount elements each.
 *  recvbufs [host array of nRanks device pointers] nRanks * sendcount each.
 *           In place: sendbufs[r] == recvbufs[r] + r * sendcount elements.
 * Same rules and transport restriction as vrReduceScatter. */
VR_API vrResult_t vrAllGather(vrComm_t comm, const void* const* sendbufs, void* const* recvbufs,
                              size_t sendcount, vrDataType_t dtype, void* stream);

/* AllReduce by the double binary tree ("NCCL 原始碼解讀", ch.4 ncclGetBtree /
 * ncclGetDtree; "NCCL 初始化流程源码级剖析", NCCL Tree 拓扑, Double Binary
 * Tree): the first alignUp(divUp(count, 2), 16/e) elements are reduced up the
 * first tree and broadcast back down it, the rest on the second tree; a node
 * combines its own element, then its first child's value, then its second
 * child's, op rounded to the element type at every step. Tree 0: rank 0 the
 * root, its child the largest power of two below N; rank r with lowest set bit
 * b under (r with bit b cleared, bit 2b set), or r - b when that is out of
 * range; children r - b/2 and r + b/2 (the second halved down while out of
 * range). Tree 1: the mirror r -> N-1-r for even N, tree 0 on ranks shifted by
 * one for odd N. The result differs from vrAllReduce's in floating-point
 * rounding (another order), not in integer or max/min results.
 * Same arguments and rules as vrAllReduce (in place allowed, count 0 returns
 * vrSuccess, nRanks 1 is a copy, sticky vrTimeout). Every rank is two warps:
 * a tree of up to 16 ranks lies in one CTA, a larger one spans the C CTAs of
 * a thread-block cluster, ceil(nRanks / C) or floor(nRanks / C) ranks in each
 * (the smallest C <= 16 leaving at most 16 ranks in each, or VR_CLUSTER_CTAS;
 * vrInvalidUsage if none). The Simple protocol
 * is used whatever the communicator's; its FIFOs live in shared memory (the
 * communicator's arena is not used). vrAvg and pre-multiplied sums scale the
 * inputs as vrAllReduce does (the integer average divides at the root). */
VR_API vrResult_t vrAllReduceTree(vrComm_t comm, const void* const* sendbufs,
                                  void* const* recvbufs, size_t count, vrDataType_t dtype,
                                  vrRedOp_t op, void* stream);

/* Calibration: the AllReduce's result without the ring. For every chunk c of
 * the ring schedule of this communicator (channels, loops of nRanks chunks of
 * chunkBytes, the last loop's chunk alignUp(divUp(rem, N), 16/e):
 * "NCCL 原始碼解讀", ch.2 §2.2-2.3), one kernel loads the N ranks' elements,
 * folds them in ring order from rank (c + 1) mod N, op(incoming, own) rounded
 * to the element type at every hop, and writes the fold to every output. The
 * result is bit for bit vrAllReduce's; the HBM traffic is the least the
 * operation allows (every input read once, every output written once), with
 * no FIFO, flag or wait. It measures the attainable ceiling of the ring
 * kernels on this GPU; it is not the ring.
 * Same arguments and rules as vrAllReduce (in place allowed, count 0 returns
 * vrSuccess), on any transport; it touches none of the communicator's FIFOs
 * and ignores its sticky timeout. */
VR_API vrResult_t vrRingWalk(vrComm_t comm, const void* const* sendbufs, void* const* recvbufs,
                             size_t count, vrDataType_t dtype, vrRedOp_t op, void* stream);

/* Wait for this communicator's outstanding work, free its memory and
 * invalidate the handle. ("NCCL 原始碼解讀", ch.1 §1.4.) Using the handle
 * afterwards returns vrInvalidArgument. */
VR_API vrResult_t vrCommDestroy(vrComm_t comm);

/* Report a device-side error found after enqueue, without synchronising
 * ("NCCL 原始碼解讀", ch.1 §1.4 ncclCommGetAsyncError). *asyncErr [out, host]
 * is vrSuccess, or vrTimeout once any wait of any kernel of this communicator
 * has given up. */
VR_API vrResult_t vrCommGetAsyncError(vrComm_t comm, vrResult_t* asyncErr);

/* Set the limit, in milliseconds (>= 1), of every device-side wait of later
 * calls on this communicator. Default 10000, or VR_TIMEOUT_MS. */
VR_API vrResult_t vrCommSetTimeout(vrComm_t comm, uint64_t timeoutMs);

/* Describe the communicator's plan (host ints written when non-NULL):
 * transport 0 = FIFOs in global memory (L2, one CTA per rank and channel;
 * VR_TRANSPORT=global), 2 = every rank a warp and every FIFO in one SM's
 * shared memory (the default for rings of 2 to 16 ranks), 3 = every rank a
 * warp, a ring spread over the C CTAs of a cluster, ceil(nRanks / C) or
 * floor(nRanks / C) ranks in each, with distributed shared memory on the CTA
 * boundaries (the default for 17 to VR_MAX_RANKS ranks); 1 is not used;
 * FIFO slot bytes and depth; device bytes the communicator allocated. */
VR_API vrResult_t vrCommGetInfo(vrComm_t comm, int* transport, int* slotBytes, int* depth,
                         size_t* deviceBytes);

/* The plan of one AllReduce of `count` elements of `dtype` on this
 * communicator, computed on the host (nothing is enqueued): *parts [out,
 * host] = the independent ring passes the call makes (per channel, loops of
 * nRanks chunks, "NCCL 原始碼解讀", ch.2 §2.2-2.3, each chunk moved in parts
 * of half the FIFO, at the FIFO geometry the call uses: on the warp
 * transports a call that needs one pass takes the smallest FIFO slot that
 * keeps it one pass, and a call that would need two or three passes takes,
 * when that saves a pass, one own-data slot per rank and the larger FIFO slot
 * it frees; results do not depend on it); *rings [out, host] = rings that run
 * at once (warp
 * transports: CTAs or clusters x rings per CTA; global: channels). A
 * ring takes its parts one after another, so ceil(parts / rings) passes of
 * 2(nRanks - 1) + 1 stages follow each other. Either pointer may be NULL.
 * vrInvalidArgument for a bad handle or dtype. */
VR_API vrResult_t vrCommGetPlan(vrComm_t comm, size_t count, vrDataType_t dtype, size_t* parts,
                                int* rings);

/* AllReduce without any allocation, for callers that cannot allocate device
 * memory where they need the collective: code under a framework's caching
 * allocator that must account for every device byte (a cudaMalloc of its own
 * could fail once the pool holds the GPU's memory, or upset its books), or a
 * latency-critical path where cudaMalloc/cudaFree would stall the device.
 * The pages have no counterpart of this call; it is this library's addition.
 * It computes exactly what a communicator created with (nRanks, nChannels,
 * proto, chunkBytes) and the global-memory FIFO transport computes, bit for
 * bit: same arguments and rules as vrAllReduce, minus the communicator, and
 * op limited to vrSum..vrMin (vrAvg and pre-multiplied sums need a
 * communicator: vrInvalidArgument).
 * Scratch (FIFOs, control words, status word) lives in one 4 MiB array that
 * the library defines in device memory; every GPU that loads the library
 * holds it until the process exits. Limits: nChannels * nRanks * 8448 + 256
 * bytes must fit in those 4 MiB (nChannels * nRanks <= 496), else
 * vrInvalidUsage; the grid (nChannels * nRanks CTAs) must be co-resident.
 * Calls allocate nothing: no cudaMalloc, cudaFree or allocating library
 * routine. The first call on each device, and the first call of each element
 * type, op and protocol on it, sets that device up (with the device current):
 * it looks up the array's device address and touches the kernel it launches.
 * Under lazy module loading (CUDA_MODULE_LOADING=LAZY, CUDA's default) that
 * set-up loads the library's modules, which reserves the 4 MiB array and
 * may allocate device memory: make those first calls before a caching pool
 * takes the GPU's memory and before any stream capture. A call with count 0
 * does the set-up and nothing else, so it serves as the warm-up. Every call
 * on a device shares the array: the call clears the part it uses
 * (cudaMemsetAsync on `stream`), so calls that overlap on the GPU (on
 * different streams, without ordering between them) race and give undefined
 * results. A device-side wait gives up after VR_TIMEOUT_MS milliseconds of
 * the environment (default 10 s); the outputs of that call are then
 * undefined and vrAllReduceNoAllocGetStatus reports vrTimeout until the next
 * call on the device clears the status. */
VR_API vrResult_t vrAllReduceNoAlloc(const void* const* sendbufs, void* const* recvbufs,
                                     size_t count, int nRanks, int nChannels, vrProto_t proto,
                                     size_t chunkBytes, vrDataType_t dtype, vrRedOp_t op,
                                     void* stream);

/* Status of the last vrAllReduceNoAlloc call on the current device, for the
 * same callers (it allocates nothing either; the pages have no counterpart).
 *  status  [out, host] vrSuccess, or vrTimeout if a device-side wait of that
 *          call gave up.
 * A synchronous read (cudaMemcpy of one word): call it after the stream of
 * the last call has been synchronised and before the next call, which clears
 * the status. vrInvalidArgument for a NULL pointer, vrCudaError if the read
 * fails. */
VR_API vrResult_t vrAllReduceNoAllocGetStatus(vrResult_t* status);

/* Create a pre-multiplied sum on `comm`: a reduction that multiplies every
 * rank's element by `scalar` (the product rounded to `dtype`; integers wrap)
 * and then sums the products in the ring's order ("NCCL 原始碼解讀", ch.6,
 * hostToDevRedOp: the host op becomes a sum whose inputs are scaled).
 *  op      [out, host] the new op, a value >= vrNumOps; unchanged on error.
 *  scalar  [host] one element of `dtype`, read during the call only.
 *  dtype   the element type the op is for: a call with another dtype returns
 *          vrInvalidArgument.
 * Valid on `comm` only, with vrAllReduce and vrReduceScatter on the on-chip
 * transports (warp, warpcluster), vrAllReduceTree and vrRingWalk; the
 * global-FIFO transport returns vrInvalidUsage for it, as it does for
 * vrAvg. At most 16 live ops per communicator (vrInvalidUsage
 * past that). */
VR_API vrResult_t vrRedOpCreatePreMulSum(vrRedOp_t* op, const void* scalar, vrDataType_t dtype,
                                         vrComm_t comm);

/* Release an op made by vrRedOpCreatePreMulSum on `comm`. vrInvalidArgument
 * for anything else. Calls already enqueued keep the scalar they were given. */
VR_API vrResult_t vrRedOpDestroy(vrRedOp_t op, vrComm_t comm);

/* ---- The operators of a data-parallel training step around the AllReduce.
 * Layer norm, whose backward pass sums the parameters' gradients over a
 * rank's rows (what the rank hands to the AllReduce), dropout, the norm and
 * rotation of query and key heads, the losses of policies and preferences with
 * their gradients, and the norm of a list
 * of gradients with clipping by it (what follows the AllReduce). They have no
 * communicator and keep nothing between calls: calls on different streams,
 * with workspaces of their own, may overlap. They are asynchronous on `stream`
 * like vrAllReduce, allocate nothing, may be captured in a CUDA graph (the
 * pointers and sizes are then those of the capture), and run on the device
 * that is current. Sums are held in 32 bits or more and added up in a fixed
 * order (no atomics), so equal calls on one GPU give equal bits; each result is
 * rounded once to its type. Outputs and workspaces overlap no other argument, except
 * where a call says so; the rows of matrices with one stride may lie side by side
 * in one buffer, those of two strides may not interleave. The pages have no
 * counterpart of them.
 * Common errors: vrInvalidArgument for a NULL or misaligned pointer (to the
 * element size; workspaces to 16 bytes), a type, size or stride outside what
 * is stated, a short workspace, or buffers that overlap where that is not
 * allowed: nothing is enqueued then. vrCudaError if a launch fails: of a call that
 * takes several launches (backward passes, long lists) the earlier ones are
 * enqueued and their outputs are written. vrInternalError if the host has no
 * memory left to check a list. */

/* Layer norm over the last axis: for each row of `cols` elements
 *   m = sum(x) / cols,  v = sum((x - m)^2) / cols,  r = 1 / sqrt(v + eps),
 *   y = (x - m) r weight + bias.
 *  x, y     [device] rows x cols of `dtype`; row i starts xStride (yStride)
 *           elements after row i - 1, strides >= cols; y's elements between
 *           cols and yStride are not written. y == x with equal strides is
 *           allowed, other overlaps are not.
 *  weight, bias  [device] cols elements of weightType each; NULL: ones, zeros.
 *  mean, rstd    [device] m and r of each row, for the backward pass; NULL:
 *           not written (inference).
 *  rows     0 returns vrSuccess and launches nothing.  cols >= 1.
 *  eps      >= 0, finite.
 *  dtype    vrFloat16, vrBfloat16 or vrFloat32; weightType: dtype or
 *           vrFloat32.
 * A NaN or infinity makes its own row NaN and no other. Every alignment and
 * stride works; rows that start on 16-byte boundaries are the fastest. */
VR_API vrResult_t vrLayerNormForward(const void* x, const void* weight, const void* bias, void* y,
                                     float* mean, float* rstd, size_t rows, size_t cols,
                                     size_t xStride, size_t yStride, float eps,
                                     vrDataType_t dtype, vrDataType_t weightType, void* stream);

/* Workspace bytes of vrLayerNormBackward for these sizes, for any strides,
 * alignments and weightType. Host only. */
VR_API vrResult_t vrLayerNormBackwardWorkspace(size_t rows, size_t cols, vrDataType_t dtype,
                                               size_t* bytes);

/* The backward pass of vrLayerNormForward: with u = (x - m) r, g = dy weight,
 *   dx = r (g - sum(g) / cols - u sum(g u) / cols)      for each row,
 *   dweight = sum over the rows of dy u,  dbias = sum over the rows of dy.
 *  dy, x, dx     [device] rows x cols of `dtype`, with row strides; dx may be
 *           NULL (only the parameters' gradients) and overlaps neither dy nor x.
 *  weight   as in the forward pass, NULL: ones.
 *  mean, rstd    [device] as the forward pass wrote them.
 *  dweight, dbias  [device] cols elements of weightType, overwritten; NULL:
 *           not wanted. With rows == 0 they become zeros.
 *  workspace     [device] 16-byte aligned, of at least
 *           vrLayerNormBackwardWorkspace bytes, used until the work on
 *           `stream` is done; may be NULL if dweight and dbias are. */
VR_API vrResult_t vrLayerNormBackward(const void* dy, const void* x, const void* weight,
                                      const float* mean, const float* rstd, void* dx,
                                      void* dweight, void* dbias, size_t rows, size_t cols,
                                      size_t dyStride, size_t xStride, size_t dxStride,
                                      vrDataType_t dtype, vrDataType_t weightType,
                                      void* workspace, size_t workspaceBytes, void* stream);

/* Workspace bytes of vrGradNorm and vrClipGradNorm for nTensors tensors of
 * any sizes. Host only. */
VR_API vrResult_t vrGradNormWorkspace(int nTensors, size_t* bytes);

/* The 2-norm of a list of gradients:
 *   norm = |scale| sqrt(sum over tensors and elements of g^2).
 *  grads    [host array of nTensors device pointers], counts [host] elements
 *           of each (0 allowed, its pointer is then not examined), dtypes
 *           [host] vrFloat16, vrBfloat16, vrFloat32 or vrFloat64 each; a list
 *           may mix them. The arrays are read during the call only.
 *  nTensors >= 1, any number.
 *  scale    finite: what the gradients are to be multiplied by (1 / nRanks
 *           after a vrSum AllReduce, or a loss scale's reciprocal).
 *  norm     [device] one float, or NULL.  tensorNorms [device] nTensors
 *           floats, each tensor's own norm, or NULL. Not both NULL.
 * Squares of float32 and bfloat16 elements that leave the range of a float
 * are summed in 64 bits; a float64 element's square has to fit a double. */
VR_API vrResult_t vrGradNorm(const void* const* grads, const size_t* counts,
                             const vrDataType_t* dtypes, int nTensors, float scale, float* norm,
                             float* tensorNorms, void* workspace, size_t workspaceBytes,
                             void* stream);

/* Clipping by the norm of the list: with norm as above,
 *   outs[t] = grads[t] * (scale * (norm > maxNorm ? maxNorm / norm : 1)),
 * in the type of grads[t], each product rounded once. The norm that decides and
 * divides is that of a double: one past the largest float (float32 elements of
 * 1e38, float64 of 1e100) still clips, while *norm, a float, is infinite. If it
 * is infinite or NaN in 64 bits as well (an element is) nothing is clipped, the
 * factor is `scale`. Read `norm` and drop the step where it is not finite.
 *  outs     [host array of nTensors device pointers]; outs[t] == grads[t] is
 *           allowed, other overlaps are not: neither with another gradient nor
 *           between two outputs (a tensor listed twice, in place).
 *  maxNorm  >= 0, may be infinite.   norm [device] one float, or NULL.
 * Other arguments as for vrGradNorm. */
VR_API vrResult_t vrClipGradNorm(const void* const* grads, void* const* outs,
                                 const size_t* counts, const vrDataType_t* dtypes, int nTensors,
                                 float scale, float maxNorm, float* norm, void* workspace,
                                 size_t workspaceBytes, void* stream);

/* Dropout by a counter-based generator, with an addition: the mask is a function of
 * the seed and of each element's number, and is never stored.
 *   y = residual + (u(n) >= round(p 2^32) ? x / (1 - p) : 0),  n = offset + row cols + column
 * u(n), 32 random bits: with block(c0, c1, c2, c3) the four words of Philox4x32-10
 * (Salmon and others, "Parallel random numbers: as easy as 1, 2, 3", 2011) under the key
 * (seed mod 2^32, seed div 2^32), and m = n div 8, the upper half is halfword n mod 8
 * (the lower half of each word first) of block(m mod 2^32, m div 2^32, 0, 0), the lower
 * half the same of block(m mod 2^32, m div 2^32, 1, 0). So a rank that passes the number
 * of its part's first element as offset drops what one rank with the whole batch drops,
 * and the backward pass is the same call on dy, without a residual.
 *  x, residual, y   [device] rows x cols of `dtype`, with row strides >= cols; residual
 *           may be NULL (nothing is added). y == x and y == residual are allowed
 *           with equal strides, other overlaps are not.
 *  p        in [0, 1]; 1 drops everything.
 *  seedDevice   [device] one uint64_t that is read by the kernel in place of `seed` (so
 *           that a captured graph draws anew each time), or NULL.
 *  offset   any; numbers wrap at 2^64.
 *  dtype    vrFloat16, vrBfloat16 or vrFloat32.
 * An element that is dropped counts for nothing, be it infinite or NaN. */
VR_API vrResult_t vrDropout(const void* x, const void* residual, void* y, size_t rows, size_t cols,
                            size_t xStride, size_t residualStride, size_t yStride, double p,
                            uint64_t seed, const uint64_t* seedDevice, uint64_t offset,
                            vrDataType_t dtype, void* stream);

/* The root-mean-square norm of each query and key head, and its rotation by the token's
 * position, in one pass: for each head x of `dim` elements
 *   r = 1 / sqrt(sum(x^2) / dim + eps),  u = x r,  y = R (u weight)
 * R turns pair i of the first rotaryDim elements, (a, b), into (a c - b s, b c + a s), with
 * c and s the elements i of row `position` of the tables. Pair i is elements i and
 * i + rotaryDim / 2, or with `interleaved` 2 i and 2 i + 1.
 *  q, k     [device] heads of `dtype`: element i of head h of token t of batch b lies
 *           at b strides[0] + t strides[1] + h strides[2] + i (strides [host], 3 each, in
 *           elements; any, 0 too). kHeads may be 0, k is then not examined.
 *  qWeight, kWeight   [device] dim elements of weightType, or NULL: ones.
 *  qOut, kOut   [device] as q and k, with strides of their own, no two elements in one
 *           place. In place (the same address and strides) is allowed, other overlaps are not.
 *  cosTable, sinTable   [device] tableRows x rotaryDim / 2 floats each.
 *  positions    [device] of positionType (vrInt32 or vrInt64), token t of batch b at
 *           b positionStride + t (0: one for all batches). The rotated elements of a
 *           token whose position is not in [0, tableRows) become NaN.
 *  batch, tokens    batch tokens < 2^31; 0 returns vrSuccess and launches nothing.
 *  dim      1 .. 1024.   rotaryDim   even, 0 .. dim; with 0 neither tables nor positions
 *           are examined.   qHeads 1 .. 65535, kHeads 0 .. 65535.
 *  eps      >= 0, finite.   dtype, weightType   as for vrLayerNormForward.
 * The sum of a head's squares has to be a float's, as that of elements below 1e17 is (beyond it
 * r is 0); a NaN or infinity reaches its own head alone. Heads whose rows start on 16-byte
 * boundaries and whose halves are whole 16 bytes are the fastest. */
VR_API vrResult_t vrQkNormRopeForward(
    const void* q, size_t qHeads, const size_t* qStrides, const void* k, size_t kHeads,
    const size_t* kStrides, const void* qWeight, const void* kWeight, void* qOut,
    const size_t* qOutStrides, void* kOut, const size_t* kOutStrides, const float* cosTable,
    const float* sinTable, size_t tableRows, const void* positions, vrDataType_t positionType,
    size_t positionStride, size_t batch, size_t tokens, size_t dim, size_t rotaryDim,
    int interleaved, float eps, vrDataType_t dtype, vrDataType_t weightType, void* stream);

/* Workspace bytes of vrQkNormRopeBackward, for any sizes. Host only. */
VR_API vrResult_t vrQkNormRopeBackwardWorkspace(size_t dim, size_t* bytes);

/* The backward pass of vrQkNormRopeForward, from its inputs: with g = R^T dy,
 *   dx = r (g weight - u sum(g weight u) / dim)      for each head,
 *   dweight = sum over tokens and heads of g u.
 *  dq, dk       [device] the gradients of qOut and kOut, dqIn, dkIn [device] those of q and
 *           k, of `dtype`, each with strides of its own; dqIn may be dq and dkIn dk with
 *           the same strides, other overlaps are not allowed.
 *  dqWeight, dkWeight   [device] dim elements of weightType, overwritten (zeros if there
 *           are no tokens, or no keys); NULL: not wanted.
 *  workspace    [device] 16-byte aligned, of at least vrQkNormRopeBackwardWorkspace bytes;
 *           may be NULL if dqWeight and dkWeight are.
 * Other arguments as in the forward pass. */
VR_API vrResult_t vrQkNormRopeBackward(
    const void* dq, const size_t* dqStrides, const void* dk, const size_t* dkStrides,
    const void* q, size_t qHeads, const size_t* qStrides, const void* k, size_t kHeads,
    const size_t* kStrides, const void* qWeight, const void* kWeight, void* dqIn,
    const size_t* dqInStrides, void* dkIn, const size_t* dkInStrides, void* dqWeight,
    void* dkWeight, const float* cosTable, const float* sinTable, size_t tableRows,
    const void* positions, vrDataType_t positionType, size_t positionStride, size_t batch,
    size_t tokens, size_t dim, size_t rotaryDim, int interleaved, float eps, vrDataType_t dtype,
    vrDataType_t weightType, void* workspace, size_t workspaceBytes, void* stream);

/* The log probability of each row's target under its logits:
 *   lse = log(sum(exp(x))),  logp = x[target] - lse
 *  logits   [device] rows x cols of `dtype` (vrFloat16, vrBfloat16, vrFloat32), row stride
 *           >= cols: what lies between cols and the stride is not read.
 *  targets  [device] one of [0, cols) a row. A negative one says that the row counts for
 *           nothing: it is not read, logp and lse are 0. One of cols or more makes logp NaN.
 *  logp, lse, rest   [device] rows floats; rest, or lse and rest, may be NULL. rest is what lse
 *           lost by being rounded: it matters where all logits of a row are large.
 *  rows     0 returns vrSuccess and launches nothing.  cols >= 1.
 * Logits of -inf are impossible tokens; +inf, NaN, or a row of -inf alone make the row NaN. */
VR_API vrResult_t vrTokenLogProbsForward(const void* logits, const int64_t* targets, float* logp,
                                         float* lse, float* rest, size_t rows, size_t cols,
                                         size_t stride, vrDataType_t dtype, void* stream);

/* The gradient of the logits from that by logp: with c = dlogp gain,
 *   dlogits[j] = c ([j = target] - exp(x[j] - lse))
 *  dlogp    [device] rows floats. A row of 0, or of a negative target, gives zeros,
 *           whatever its logits hold; they are not read.
 *  gain     [device] one float, or NULL: 1.
 *  lse, rest    [device] as the forward pass wrote them; rest NULL: zeros.
 *  dlogits  [device] rows x cols of `dtype`, row stride dStride; may be logits, with the
 *           same stride; other overlaps are not allowed. */
VR_API vrResult_t vrTokenLogProbsBackward(const float* dlogp, const float* gain,
                                          const void* logits, const int64_t* targets,
                                          const float* lse, const float* rest, void* dlogits,
                                          size_t rows, size_t cols, size_t stride, size_t dStride,
                                          vrDataType_t dtype, void* stream);

/* Workspace bytes of vrPolicyLoss. Host only. */
VR_API vrResult_t vrPolicyLossWorkspace(size_t rows, size_t* bytes);

/* The clipped loss of a policy with a term that holds it to a reference policy, and its
 * gradient: with logp as above and e = logp - oldLogp, a row's loss is
 *   -min(exp(e) A, min(max(exp(e), 1 - clipLow), 1 + clipHigh) A)
 *     + klCoef (exp(refLogp - logp) - (refLogp - logp) - 1)
 * and loss = scale sum(weight times the row's loss). Where the clipped ratio decides the
 * first term has no derivative.
 *  oldLogp, advantages (A)   [device] rows floats. The first term of a row of advantage 0 is 0,
 *           but NaN where e is: broken logits, or a target that is none, are not hidden.
 *  weights  [device] rows floats, or NULL: ones. A row of weight 0, or of a negative
 *           target, counts for nothing, whatever its other inputs hold.
 *  refLogp  [device] rows floats, or NULL: no such term; nor is there one if klCoef is 0. Where
 *           refLogp - logp is infinite, either way, so is the term.
 *  loss     [device] one float. 0 without rows.
 *  logp, lse, rest, dlogp   [device] rows floats: the last is the loss's derivative by logp, for
 *           vrTokenLogProbsBackward. Rows that count for nothing get zeros in all of them.
 *  dlogits  [device] the gradient of the logits, or NULL: not wanted. May be logits, as in
 *           vrTokenLogProbsBackward.
 *  clipLow, clipHigh    >= 0, may be infinite.   klCoef, scale   finite.
 *  workspace    [device] 16-byte aligned, of at least vrPolicyLossWorkspace bytes. */
VR_API vrResult_t vrPolicyLoss(const void* logits, const int64_t* targets, const float* oldLogp,
                               const float* advantages, const float* weights,
                               const float* refLogp, float* loss, float* logp, float* lse,
                               float* rest, float* dlogp, void* dlogits, size_t rows, size_t cols,
                               size_t stride, size_t dStride, double clipLow, double clipHigh,
                               float klCoef, float scale, vrDataType_t dtype, void* workspace,
                               size_t workspaceBytes, void* stream);

/* Workspace bytes of vrPreferenceLoss. Host only. */
VR_API vrResult_t vrPreferenceLossWorkspace(size_t pairs, size_t* bytes);

/* The loss of preferences between paired sequences, by the ratio of their probabilities
 * under the policy to those under a reference, and its gradient. Sequence s < pairs is
 * pair s's chosen one, pairs + s its rejected one; S is the sum of logp over a sequence's rows.
 *   h = beta ((S - ref)[chosen] - (S - ref)[rejected])
 *   loss = scale sum over pairs of (1 - labelSmoothing) log(1 + exp(-h)) + labelSmoothing log(1 + exp(h))
 * A term whose factor is 0 is left out: an impossible token (a target's logit of -inf) in one of
 * a pair's sequences makes h infinite and the pair's loss 0 or infinite, not NaN; in both, NaN.
 *  starts   [device] 2 pairs + 1 numbers of rows: sequence s is the rows from starts[s] to
 *           before starts[s + 1], cut at the rows that there are; none where the second is
 *           not larger. Rows of no sequence count for nothing. They do not decrease: where
 *           they do and a row is in two sequences, its derivative is that of either.
 *           NULL: the rows in 2 pairs equal parts.
 *  targets  negative: the row (of a prompt, or padding) counts for nothing.
 *  refLogps     [device] 2 pairs floats, or NULL: zeros.
 *  loss     [device] one float.  logps   [device] 2 pairs floats, S.
 *  logp, lse, rest, dlogp, dlogits   as in vrPolicyLoss, but that logp, lse and rest of rows
 *           of no sequence are theirs.
 *  pairs >= 1, rows any.  beta, scale   finite.  labelSmoothing   in [0, 1].
 *  workspace    [device] 16-byte aligned, of at least vrPreferenceLossWorkspace bytes. */
VR_API vrResult_t vrPreferenceLoss(const void* logits, const int64_t* targets,
                                   const float* refLogps, const int64_t* starts, float* loss,
                                   float* logps, float* logp, float* lse, float* rest, float* dlogp,
                                   void* dlogits, size_t pairs, size_t rows, size_t cols,
                                   size_t stride, size_t dStride, float beta,
                                   float labelSmoothing, float scale, vrDataType_t dtype,
                                   void* workspace, size_t workspaceBytes, void* stream);

/* Static description of a result code. Never NULL. */
VR_API const char* vrGetErrorString(vrResult_t result);

#ifdef __cplusplus
}
#endif

#endif /* VR_H_ */
