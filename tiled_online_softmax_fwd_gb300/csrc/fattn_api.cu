// fattn_api.cu -- the C ABI of libfattn (see include/fattn.h).
//
// Validation follows the wrapper conventions of "Triton programming
// template" (check device, shape, dtype and layout before launching; return
// early for empty inputs; launch asynchronously on the caller's stream).  All
// checks are synchronous and nothing is enqueued when one fails.
#include <cudaTypedefs.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "fattn.h"
#include "fattn_internal.h"

namespace {

thread_local int t_last_cuda_error = 0;

fattn_status_t cuda_fail(cudaError_t e)
{
    t_last_cuda_error = static_cast<int>(e);
    return FATTN_ERR_CUDA;
}

// Per-device facts, read once.
struct DeviceInfo {
    bool probed = false;
    bool supported = false;
    int num_sms = 0;
    int dev = -1;
};
constexpr int kMaxDevices = 64;
std::mutex g_dev_mutex;
DeviceInfo g_dev[kMaxDevices];

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;
cudaError_t g_encode_err = cudaSuccess;

fattn_status_t current_device(int *dev, DeviceInfo *info)
{
    cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess)
        return cuda_fail(e);
    if (*dev < 0 || *dev >= kMaxDevices)
        return FATTN_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(g_dev_mutex);
    DeviceInfo &d = g_dev[*dev];
    if (!d.probed) {
        int major = 0, minor = 0, sms = 0;
        if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, *dev)) != cudaSuccess)
            return cuda_fail(e);
        d.supported = (major == 10 && minor == 3);  // the kernels are built for sm_103a only
        d.num_sms = sms;
        d.dev = *dev;
        d.probed = true;
    }
    *info = d;
    return d.supported ? FATTN_OK : FATTN_ERR_UNSUPPORTED;
}

fattn_status_t get_encoder(PFN_cuTensorMapEncodeTiled_v12000 *fn)
{
    std::call_once(g_encode_once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        g_encode_err = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                        cudaEnableDefault, &q);
        if (g_encode_err == cudaSuccess && q != cudaDriverEntryPointSuccess)
            g_encode_err = cudaErrorSymbolNotFound;
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    if (g_encode_err != cudaSuccess || g_encode == nullptr)
        return cuda_fail(g_encode_err != cudaSuccess ? g_encode_err : cudaErrorSymbolNotFound);
    *fn = g_encode;
    return FATTN_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Shape and scalar checks that need no device.  Sets *empty when there is no
// work (B*H*N == 0).
fattn_status_t check_shape(int B, int H, int N, int d, float scale, int causal, bool *empty)
{
    if (B < 0 || H < 0 || N < 0)
        return FATTN_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1)
        return FATTN_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !isfinite(scale))
        return FATTN_ERR_INVALID_ARG;
    if (d != 64 && d != 96 && d != 128 && d != 256)
        return FATTN_ERR_UNSUPPORTED;
    const long long rows = static_cast<long long>(B) * H * N;
    *empty = rows == 0;
    // Each tensor must stay below 2^40 bytes (tensor-map stride limit) and
    // B*H must fit the tensor map's outer dimension.
    if (static_cast<long long>(B) * H > 0x7fffffffLL)
        return FATTN_ERR_UNSUPPORTED;
    if (!*empty && rows > (1LL << 39) / (2LL * d))
        return FATTN_ERR_UNSUPPORTED;
    return FATTN_OK;
}

// Key-length checks of a call whose keys (Nk) may differ from its queries
// (Nq): Nk >= 0, at least one key when there are queries, Nq <= Nk under the
// causal mask (the queries are the last Nq key positions), and K, V within the
// same size limit as Q.
fattn_status_t check_keys(int B, int H, int Nq, int Nk, int d, int causal)
{
    if (Nk < 0)
        return FATTN_ERR_INVALID_ARG;
    const long long q_rows = static_cast<long long>(B) * H * Nq;
    if (q_rows > 0 && Nk == 0)
        return FATTN_ERR_INVALID_ARG;
    if (causal && Nq > Nk)
        return FATTN_ERR_INVALID_ARG;
    if (q_rows > 0 && static_cast<long long>(B) * H * Nk > (1LL << 39) / (2LL * d))
        return FATTN_ERR_UNSUPPORTED;
    return FATTN_OK;
}

// Pointer checks: non-null, 16-byte aligned, no output overlapping an input or
// the other output.  q_bytes covers q and o, kv_bytes each of k and v.
fattn_status_t check_pointers(const void *q, const void *k, const void *v, const void *o,
                              const float *lse, size_t q_bytes, size_t kv_bytes, size_t lse_bytes)
{
    if (!q || !k || !v || !o || !lse)
        return FATTN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return FATTN_ERR_INVALID_ARG;
    if (overlap(o, q_bytes, q, q_bytes) || overlap(o, q_bytes, k, kv_bytes) ||
        overlap(o, q_bytes, v, kv_bytes) || overlap(o, q_bytes, lse, lse_bytes) ||
        overlap(lse, lse_bytes, q, q_bytes) || overlap(lse, lse_bytes, k, kv_bytes) ||
        overlap(lse, lse_bytes, v, kv_bytes))
        return FATTN_ERR_INVALID_ARG;
    return FATTN_OK;
}

// The buffer must be device (or managed) memory of the current device.
fattn_status_t check_device_buffer(const void *p, int dev)
{
    cudaPointerAttributes attr;
    cudaError_t e = cudaPointerGetAttributes(&attr, p);
    if (e != cudaSuccess) {
        cudaGetLastError();  // clear the sticky-free error state of this query
        return FATTN_ERR_INVALID_ARG;
    }
    if (attr.type == cudaMemoryTypeDevice)
        return attr.device == dev ? FATTN_OK : FATTN_ERR_INVALID_ARG;
    if (attr.type == cudaMemoryTypeManaged)
        return FATTN_OK;
    return FATTN_ERR_INVALID_ARG;
}

fattn_status_t make_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap *m, const void *ptr,
                        int N, int d, long long BH, bool f16 = false)
{
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N),
                                static_cast<cuuint64_t>(BH)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2,
                                   static_cast<cuuint64_t>(N) * static_cast<cuuint64_t>(d) * 2};
    const cuuint32_t box[3] = {64, 128, 1};
    const cuuint32_t elem_strides[3] = {1, 1, 1};
    const CUresult r = encode(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                              3, const_cast<void *>(ptr), dims,
                              strides, box, elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        t_last_cuda_error = static_cast<int>(r);
        return FATTN_ERR_CUDA;
    }
    return FATTN_OK;
}

// Element strides (batch, head, row) of q, k, v and o; the last dimension
// (d) is contiguous.
struct Layout {
    long long q[3], k[3], v[3], o[3];
};

Layout dense_layout(int H, int N, int Nk, int d)
{
    const long long qn = d, qh = static_cast<long long>(N) * d, qb = qh * H;
    const long long kh = static_cast<long long>(Nk) * d, kb = kh * H;
    return Layout{{qb, qh, qn}, {kb, kh, qn}, {kb, kh, qn}, {qb, qh, qn}};
}

// Bytes from a tensor's base to one past its last element.
size_t span_bytes(const long long st[3], int B, int H, int rows, int d)
{
    return static_cast<size_t>(st[0] * (B - 1) + st[1] * (H - 1) +
                               st[2] * static_cast<long long>(rows - 1) + d) * 2;
}

// 4-D map (d, rows, H, B) of a 16-bit tensor with element strides st
// (batch, head, row), box (64, box_rows, 1, 1), 128-byte swizzle, zero fill
// outside the tensor.  box_rows is 128 (one tile's rows), or 64 for V at
// d = 256, whose kernel copies each V tile as two halves of 64 keys.
fattn_status_t make_map4(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap *m,
                         const void *ptr, int rows, int d, int H, int B, const long long st[3],
                         bool f16, unsigned box_rows = 128)
{
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(B)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(st[2]) * 2,
                                   static_cast<cuuint64_t>(st[1]) * 2,
                                   static_cast<cuuint64_t>(st[0]) * 2};
    const cuuint32_t box[4] = {64, box_rows, 1, 1};
    const cuuint32_t elem_strides[4] = {1, 1, 1, 1};
    const CUresult r = encode(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                              4, const_cast<void *>(ptr), dims, strides, box, elem_strides,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        t_last_cuda_error = static_cast<int>(r);
        return FATTN_ERR_CUDA;
    }
    return FATTN_OK;
}

// Stride rules of a strided call: every stride a positive multiple of 8
// elements (16 bytes, the tensor-map rule; o is written in 16-byte pieces),
// each tensor's span below 2^39 bytes, o's elements all distinct (nested
// strides: sorted by size, each stride at least the span of the smaller
// dimensions), and no output overlapping an input or the other output.
fattn_status_t check_layout(const void *q, const void *k, const void *v, const void *o,
                            const float *lse, int B, int H, int N, int Nk, int d, const Layout &L)
{
    if (!q || !k || !v || !o || !lse)
        return FATTN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return FATTN_ERR_INVALID_ARG;
    const long long *all[4] = {L.q, L.k, L.v, L.o};
    const int rows[4] = {N, Nk, Nk, N};
    size_t span[4];
    for (int t = 0; t < 4; ++t) {
        for (int i = 0; i < 3; ++i)
            if (all[t][i] < 1 || all[t][i] % 8 != 0 || all[t][i] > (1LL << 38))
                return FATTN_ERR_INVALID_ARG;
        const long double far = static_cast<long double>(all[t][0]) * (B - 1) +
                                static_cast<long double>(all[t][1]) * (H - 1) +
                                static_cast<long double>(all[t][2]) * (rows[t] - 1) + d;
        if (far * 2 >= static_cast<long double>(1LL << 39))
            return FATTN_ERR_UNSUPPORTED;
        span[t] = span_bytes(all[t], B, H, rows[t], d);
    }
    // o: nested strides over the dimensions of extent > 1.
    long long st[3] = {L.o[2], L.o[1], L.o[0]};
    long long ext[3] = {N, H, B};
    for (int i = 0; i < 3; ++i)  // sort by stride (3 elements)
        for (int j = i + 1; j < 3; ++j)
            if (st[j] < st[i]) {
                long long t = st[i]; st[i] = st[j]; st[j] = t;
                t = ext[i]; ext[i] = ext[j]; ext[j] = t;
            }
    long long covered = d;
    for (int i = 0; i < 3; ++i) {
        if (ext[i] <= 1)
            continue;
        if (st[i] < covered)
            return FATTN_ERR_INVALID_ARG;
        covered += st[i] * (ext[i] - 1);
    }
    const size_t lb = static_cast<size_t>(B) * H * N * 4;
    if (overlap(o, span[3], q, span[0]) || overlap(o, span[3], k, span[1]) ||
        overlap(o, span[3], v, span[2]) || overlap(o, span[3], lse, lb) ||
        overlap(lse, lb, q, span[0]) || overlap(lse, lb, k, span[1]) ||
        overlap(lse, lb, v, span[2]))
        return FATTN_ERR_INVALID_ARG;
    return FATTN_OK;
}

// kTcgen05: bf16, P in fp16 (V converted on chip); kTcgen05F16: fp16;
// kTcgen05Bf16P: bf16, P in bf16; kSimt: the fp32 cross-check kernel.
enum class Kernel { kTcgen05, kTcgen05F16, kTcgen05Bf16P, kSimt };

// Every check of a forward call with N queries and Nk keys per head.  On
// FATTN_OK, *empty tells whether there is any work, and (when there is)
// *dev / *info describe the current device.
// L == nullptr: contiguous tensors.
fattn_status_t validate(const void *q, const void *k, const void *v, const void *o,
                        const float *lse, int B, int H, int N, int Nk, int d, float scale,
                        int causal, bool *empty, int *dev, DeviceInfo *info,
                        const Layout *L = nullptr)
{
    fattn_status_t s = check_shape(B, H, N, d, scale, causal, empty);
    if (s != FATTN_OK)
        return s;
    if ((s = check_keys(B, H, N, Nk, d, causal)) != FATTN_OK || *empty)
        return s;
    const size_t rows = static_cast<size_t>(B) * H * N;
    const size_t kv_bytes = static_cast<size_t>(B) * H * Nk * d * 2;
    if (L != nullptr)
        s = check_layout(q, k, v, o, lse, B, H, N, Nk, d, *L);
    else
        s = check_pointers(q, k, v, o, lse, rows * d * 2, kv_bytes, rows * 4);
    if (s != FATTN_OK)
        return s;
    if ((s = current_device(dev, info)) != FATTN_OK)
        return s;
    const void *bufs[5] = {q, k, v, o, lse};
    for (const void *p : bufs)
        if ((s = check_device_buffer(p, *dev)) != FATTN_OK)
            return s;
    return FATTN_OK;
}

// ---------------------------------------------------------------- V pre-pass
// For bf16 inputs with P in fp16, V is rounded to fp16 either on chip, per
// work unit, by the forward kernel's converter warps, or once per call by a
// pre-pass into scratch that the forward kernel then reads (the same bits
// either way).  The scratch comes from one stream-ordered memory pool per
// device, created on first use, which keeps freed blocks for the next call
// (release threshold: unlimited), so a steady loop of calls maps no new
// device memory; fattn_trim_scratch returns them.
std::atomic<int> g_v_convert{FATTN_V_CONVERT_AUTO};
std::mutex g_pool_mutex;
cudaMemPool_t g_pool[kMaxDevices] = {};

// FATTN_V_CONVERT_AUTO: the pre-pass where it was measured to pay.  The
// converter warps round each V tile once for every work unit that reads it
// (a pair of 128-row Q tiles, one Q tile at d = 256), on average `visits`
// times: the units per head, halved under the causal mask.  The pre-pass
// costs a fixed 4 bytes of HBM traffic per V element and one more launch.
// On one GB300 (bf16, L2 flushed) it was faster from these visits on and
// slower below them: d = 64 from 24 (16: -0.4 %, 24: +2 %, 256: +4 %);
// d = 96 from 8 (4: -3 % to +1 %, 8: +4.5 %); d = 128 from 16 (12: -1.5 %,
// 16: +0.6 % causal and +3 % not, 32: +3 to +5 %); d = 256 from 12 (8: -1 %
// to -6 %, 12: +13 %, 32: +36 %).
enum class VRoute { kOnChip, kPrepass };

VRoute v_route(int Nq, int d, int causal)
{
    if (Nq <= 0)
        return VRoute::kOnChip;
    const int mode = g_v_convert.load(std::memory_order_relaxed);
    if (mode == FATTN_V_CONVERT_PREPASS)
        return VRoute::kPrepass;
    if (mode == FATTN_V_CONVERT_ON_CHIP)
        return VRoute::kOnChip;
    const long long tiles = (static_cast<long long>(Nq) + 127) / 128;
    const long long units = d == 256 ? tiles : (tiles + 1) / 2;
    const long long visits2 = causal ? units : 2 * units;  // twice the visits
    const long long need2 = d == 64 ? 48 : d == 96 ? 16 : d == 128 ? 32 : 24;
    return visits2 >= need2 ? VRoute::kPrepass : VRoute::kOnChip;
}


// Scratch of `bytes` on `stream`, or nullptr where there is none to be had
// (the stream is being captured into a graph, the pool cannot be created or
// the device is out of memory): the caller then converts on chip.
void *prepass_scratch(int dev, size_t bytes, cudaStream_t stream)
{
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(stream, &cs) != cudaSuccess || cs != cudaStreamCaptureStatusNone) {
        cudaGetLastError();
        return nullptr;
    }
    cudaMemPool_t pool = nullptr;
    {
        std::lock_guard<std::mutex> lock(g_pool_mutex);
        if (g_pool[dev] == nullptr) {
            cudaMemPoolProps props = {};
            props.allocType = cudaMemAllocationTypePinned;
            props.handleTypes = cudaMemHandleTypeNone;
            props.location.type = cudaMemLocationTypeDevice;
            props.location.id = dev;
            cudaMemPool_t created = nullptr;
            if (cudaMemPoolCreate(&created, &props) != cudaSuccess) {
                cudaGetLastError();
                return nullptr;
            }
            uint64_t keep = UINT64_MAX;
            cudaMemPoolSetAttribute(created, cudaMemPoolAttrReleaseThreshold, &keep);
            g_pool[dev] = created;
        }
        pool = g_pool[dev];
    }
    void *ptr = nullptr;
    if (cudaMallocFromPoolAsync(&ptr, bytes, pool, stream) != cudaSuccess) {
        cudaGetLastError();
        return nullptr;
    }
    return ptr;
}

// Enqueue one validated forward call with N queries and Nk keys per head
// (split.splits > 1: key-range split with the caller's scratch).
// may_allocate false: no device memory is taken (V is converted on chip).
fattn_status_t launch(Kernel which, const DeviceInfo &info, const void *q, const void *k,
                      const void *v, void *o, float *lse, int B, int H, int N, int Nk, int d,
                      float scale, int causal, cudaStream_t stream,
                      const fattn::FwdSplit &split = fattn::FwdSplit{1, nullptr, nullptr},
                      const Layout *L = nullptr, bool may_allocate = true)
{
    fattn::FwdArgs a{q, k, v, o, lse, B, H, N, d, scale, causal};
    const bool f16 = which == Kernel::kTcgen05F16;
    a.f16 = f16 ? 1 : 0;
    a.bf16p = which == Kernel::kTcgen05Bf16P ? 1 : 0;
    a.Nk = Nk;
    cudaError_t e;
    if (which == Kernel::kSimt) {
        if (Nk != N || L != nullptr || d > 128)
            return FATTN_ERR_UNSUPPORTED;
        e = fattn::launch_fwd_simt(a, stream);
    } else {
        PFN_cuTensorMapEncodeTiled_v12000 encode;
        fattn_status_t s;
        if ((s = get_encoder(&encode)) != FATTN_OK)
            return s;
        const Layout lay = L != nullptr ? *L : dense_layout(H, N, Nk, d);
        a.o_sb = lay.o[0];
        a.o_sh = lay.o[1];
        a.o_sn = lay.o[2];
        fattn::FwdMaps maps;
        if ((s = make_map4(encode, &maps.q, q, N, d, H, B, lay.q, f16)) != FATTN_OK ||
            (s = make_map4(encode, &maps.k, k, Nk, d, H, B, lay.k, f16)) != FATTN_OK)
            return s;
        void *v16 = nullptr;
        const unsigned v_box_rows = d == 256 ? 64u : 128u;
        if (which == Kernel::kTcgen05 && may_allocate && v_route(N, d, causal) == VRoute::kPrepass)
            v16 = prepass_scratch(info.dev, static_cast<size_t>(B) * H * Nk * d * 2, stream);
        if (v16 != nullptr) {
            const Layout dense = dense_layout(H, N, Nk, d);
            a.v16 = v16;
            a.v_sb = lay.v[0];
            a.v_sh = lay.v[1];
            a.v_sn = lay.v[2];
            s = make_map4(encode, &maps.v, v16, Nk, d, H, B, dense.v, true, v_box_rows);
        } else {
            s = make_map4(encode, &maps.v, v, Nk, d, H, B, lay.v, f16, v_box_rows);
        }
        e = s == FATTN_OK ? fattn::launch_fwd_sm103(a, maps, split, info.num_sms, stream)
                          : cudaSuccess;
        if (v16 != nullptr) {
            const cudaError_t ef = cudaFreeAsync(v16, stream);
            if (e == cudaSuccess)
                e = ef;
        }
        if (s != FATTN_OK)
            return s;
    }
    return e == cudaSuccess ? FATTN_OK : cuda_fail(e);
}

fattn_status_t forward(Kernel which, const void *q, const void *k, const void *v, void *o,
                       float *lse, int B, int H, int N, int d, float scale, int causal,
                       cudaStream_t stream, bool may_allocate = true)
{
    bool empty = false;
    int dev = 0;
    DeviceInfo info;
    fattn_status_t s =
        validate(q, k, v, o, lse, B, H, N, N, d, scale, causal, &empty, &dev, &info);
    if (s != FATTN_OK || empty)
        return s;
    return launch(which, info, q, k, v, o, lse, B, H, N, N, d, scale, causal, stream,
                  fattn::FwdSplit{1, nullptr, nullptr}, nullptr, may_allocate);
}

constexpr int kMaxSplits = 64;
constexpr size_t kWsAlign = 256;


// Scratch layout of a split call: fp32 partial O, then (256-byte aligned) the
// base-2 partial lse pairs.
size_t split_ws_o_bytes(int B, int H, int N, int d, int splits)
{
    return static_cast<size_t>(splits) * B * H * N * d * sizeof(float);
}
size_t split_ws_bytes(int B, int H, int N, int d, int splits)
{
    if (splits <= 1)
        return 0;
    return align_up(split_ws_o_bytes(B, H, N, d, splits), kWsAlign) +
           static_cast<size_t>(splits) * B * H * N * 2 * sizeof(float);
}

// Splits for a grid of fewer work units than SMs: the s (at most one split
// per two key tiles, at most kMaxSplits) that minimises the estimated time in
// key-tile steps: ceil(units * s / SMs) rounds of ceil(KT / s) steps plus
// kUnitCost steps per unit (Q load, pipeline fill, epilogue), plus
// kMergeCost steps for the partial outputs and their merge when s > 1 (both
// measured on one and four splits of 16 pairs x 32 key tiles, d = 64).  Ties
// go to the smaller s.
constexpr long long kUnitCost = 3, kMergeCost = 6;
int choose_splits(int B, int H, int Nq, int Nk, int d, int num_sms)
{
    // A work unit is a pair of 128-row Q tiles, or one Q tile for d = 256.
    const long long q_tiles = (static_cast<long long>(Nq) + 127) / 128;
    const long long pairs = d == 256 ? q_tiles : (q_tiles + 1) / 2;
    const long long units = static_cast<long long>(B) * H * pairs;
    const long long key_tiles = (static_cast<long long>(Nk) + 127) / 128;
    if (units <= 0 || units >= num_sms)
        return 1;
    long long best_s = 1, best = key_tiles + kUnitCost;
    const long long s_max = key_tiles / 2 < kMaxSplits ? key_tiles / 2 : kMaxSplits;
    for (long long s = 2; s <= s_max; ++s) {
        const long long rounds = (units * s + num_sms - 1) / num_sms;
        const long long est = rounds * ((key_tiles + s - 1) / s + kUnitCost) + kMergeCost;
        if (est < best) {
            best = est;
            best_s = s;
        }
    }
    return static_cast<int>(best_s);
}

// The automatic schedule of attn_fwd_kv: stream-K for one Q-tile pair per
// head when whole heads would leave SMs idle, else choose_splits.  Returns
// the partial slots per head (1: no split).
int auto_slots(int B, int H, int Nq, int Nk, int d, int causal, int num_sms, int *streamk)
{
    const fattn::FwdPlan plan = fattn::plan_fwd_streamk(B, H, Nq, Nk, causal, num_sms);
    *streamk = plan.streamk;
    return plan.streamk ? plan.slots : choose_splits(B, H, Nq, Nk, d, num_sms);
}

// num_splits == 0: the automatic schedule for the current device.
// L == nullptr: contiguous tensors.
fattn_status_t forward_split(const void *q, const void *k, const void *v, void *o, float *lse,
                             int B, int H, int N, int Nk, int d, float scale, int causal,
                             int num_splits, void *workspace, size_t workspace_bytes,
                             cudaStream_t stream, const Layout *L = nullptr,
                             Kernel which = Kernel::kTcgen05, bool may_allocate = true)
{
    if (num_splits < 0 || num_splits > kMaxSplits)
        return FATTN_ERR_INVALID_ARG;
    bool empty = false;
    int dev = 0;
    DeviceInfo info;
    fattn_status_t s =
        validate(q, k, v, o, lse, B, H, N, Nk, d, scale, causal, &empty, &dev, &info, L);
    if (s != FATTN_OK || empty)
        return s;
    int streamk = 0;
    if (num_splits == 0)
        num_splits = auto_slots(B, H, N, Nk, d, causal, info.num_sms, &streamk);
    if (num_splits == 1)
        return launch(which, info, q, k, v, o, lse, B, H, N, Nk, d, scale, causal, stream,
                      fattn::FwdSplit{1, nullptr, nullptr}, L, may_allocate);
    const size_t need = split_ws_bytes(B, H, N, d, num_splits);
    if (!workspace || !aligned16(workspace) || workspace_bytes < need)
        return FATTN_ERR_INVALID_ARG;
    const Layout lay = L != nullptr ? *L : dense_layout(H, N, Nk, d);
    const size_t lb = static_cast<size_t>(B) * H * N * 4;
    if (overlap(workspace, need, q, span_bytes(lay.q, B, H, N, d)) ||
        overlap(workspace, need, k, span_bytes(lay.k, B, H, Nk, d)) ||
        overlap(workspace, need, v, span_bytes(lay.v, B, H, Nk, d)) ||
        overlap(workspace, need, o, span_bytes(lay.o, B, H, N, d)) ||
        overlap(workspace, need, lse, lb))
        return FATTN_ERR_INVALID_ARG;
    if ((s = check_device_buffer(workspace, dev)) != FATTN_OK)
        return s;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const fattn::FwdSplit split{
        num_splits, reinterpret_cast<float *>(ws),
        reinterpret_cast<float *>(ws + align_up(split_ws_o_bytes(B, H, N, d, num_splits), kWsAlign)),
        streamk};
    return launch(which, info, q, k, v, o, lse, B, H, N, Nk, d, scale, causal, stream, split, L,
                  may_allocate);
}

// ---------------------------------------------------------------- no-allocation split
// Scratch for attn_fwd_split_noalloc: a fixed device array that lives as long
// as the library is loaded, so that callers that may not allocate device
// memory on their execution path still get the split kernel.  Its device
// address is looked up once per device (cudaGetSymbolAddress, with that device
// current); in host code the array's name is only a host-side stand-in.
constexpr size_t kNoAllocScratchBytes = size_t(32) << 20;
__device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

std::mutex g_noalloc_mutex;
void *g_noalloc_ptr[kMaxDevices] = {};

fattn_status_t noalloc_scratch(int dev, void **out)
{
    std::lock_guard<std::mutex> lock(g_noalloc_mutex);
    if (g_noalloc_ptr[dev] == nullptr) {
        void *ptr = nullptr;
        const cudaError_t e = cudaGetSymbolAddress(&ptr, g_noalloc_scratch);
        if (e != cudaSuccess || ptr == nullptr)
            return cuda_fail(e != cudaSuccess ? e : cudaErrorInvalidSymbol);
        g_noalloc_ptr[dev] = ptr;
    }
    *out = g_noalloc_ptr[dev];
    return FATTN_OK;
}

// attn_fwd_host's copy/compute pipeline: per-device helper streams and
// events, created on first use and kept for the process.  Calls are
// serialised by g_pipe_mutex (each call synchronises before it returns).
constexpr int kHostChunks = 16;

// Head ranges [bounds[c], bounds[c+1]) of that pipeline.  Nothing overlaps
// the first chunk's copy in, nor the last chunk's kernel and copy out, so the
// ends are kept short: chunks of m/4 and m/2 heads first, equal chunks of
// about m = ceil(BH/8) in the middle, m/2 and m/4 last.  No chunk has fewer
// than min_heads heads, the heads that give every SM a work unit: a chunk's
// kernel lasts at least as long as its heaviest unit, so smaller chunks would
// only leave SMs idle.  Shapes too small for the ramps get equal chunks.
// Returns the number of chunks (at most 11).
int host_chunk_plan(long long BH, long long min_heads, long long bounds[kHostChunks + 1])
{
    const long long m = std::max((BH + 7) / 8, min_heads);
    const long long q = std::max(m / 4, min_heads), h = std::max(m / 2, min_heads);
    const long long rest = BH - 2 * (q + h);
    int n = 0;
    bounds[0] = 0;
    if (rest < m) {
        n = static_cast<int>(std::min<long long>((BH + m - 1) / m, 8));
        for (int c = 1; c <= n; ++c)
            bounds[c] = BH * c / n;
        return n;
    }
    const long long k = rest / m;  // middle chunks, 1..7
    for (long long sz : {q, h})
        bounds[n + 1] = bounds[n] + sz, ++n;
    for (long long i = 0; i < k; ++i)
        bounds[n + 1] = bounds[n] + rest / k + (i < rest % k ? 1 : 0), ++n;
    for (long long sz : {h, q})
        bounds[n + 1] = bounds[n] + sz, ++n;
    return n;
}
struct HostPipe {
    bool ready = false;
    cudaStream_t in = nullptr, out = nullptr;
    cudaEvent_t start = nullptr;
    cudaEvent_t ev_in[kHostChunks] = {}, ev_done[kHostChunks] = {};
};
std::mutex g_pipe_mutex;
HostPipe g_pipe[kMaxDevices];

fattn_status_t host_pipe(int dev, HostPipe **out)
{
    HostPipe &hp = g_pipe[dev];
    if (!hp.ready) {
        cudaError_t e = cudaStreamCreateWithFlags(&hp.in, cudaStreamNonBlocking);
        if (e == cudaSuccess)
            e = cudaStreamCreateWithFlags(&hp.out, cudaStreamNonBlocking);
        if (e == cudaSuccess)
            e = cudaEventCreateWithFlags(&hp.start, cudaEventDisableTiming);
        for (int c = 0; c < kHostChunks && e == cudaSuccess; ++c) {
            e = cudaEventCreateWithFlags(&hp.ev_in[c], cudaEventDisableTiming);
            if (e == cudaSuccess)
                e = cudaEventCreateWithFlags(&hp.ev_done[c], cudaEventDisableTiming);
        }
        if (e != cudaSuccess)
            return cuda_fail(e);
        hp.ready = true;
    }
    *out = &hp;
    return FATTN_OK;
}

// ---------------------------------------------------------------- row sets
// One strided tensor of 16-bit rows of d elements: base, element strides and
// extents of its outer dimensions (unused ones have extent 1).
struct Rows {
    const void *p;
    long long st[3];
    long long ext[3];
    int d;
};

Rows rows_of(const void *p, const long long *st, int n_dims, long long e0, long long e1,
             long long e2, int d)
{
    Rows r{p, {1, 1, 1}, {e0, e1, n_dims > 2 ? e2 : 1}, d};
    for (int i = 0; i < n_dims; ++i)
        r.st[i] = st[i];
    return r;
}

bool empty(const Rows &r) { return r.ext[0] == 0 || r.ext[1] == 0 || r.ext[2] == 0; }

// Elements from the base to one past the last.
long long extent_of(const Rows &r)
{
    long long n = r.d;
    for (int i = 0; i < 3; ++i)
        n += r.st[i] * (r.ext[i] - 1);
    return n;
}

// Alignment and stride rules: base 16-byte aligned; each stride of a
// dimension of extent > 1 a positive multiple of 8 elements, at most 2^38;
// the span below 2^39 bytes.
fattn_status_t check_rows(const Rows &r)
{
    if (!r.p || !aligned16(r.p))
        return FATTN_ERR_INVALID_ARG;
    long double far = r.d;
    for (int i = 0; i < 3; ++i) {
        if (r.ext[i] <= 1)
            continue;
        if (r.st[i] < 1 || r.st[i] % 8 != 0 || r.st[i] > (1LL << 38))
            return FATTN_ERR_INVALID_ARG;
        far += static_cast<long double>(r.st[i]) * (r.ext[i] - 1);
    }
    return far * 2 >= static_cast<long double>(1LL << 39) ? FATTN_ERR_UNSUPPORTED : FATTN_OK;
}

// Whether all elements are distinct, by nesting: the strides sorted by size,
// each at least the span of the smaller dimensions.
bool distinct(const Rows &r)
{
    int at[3] = {0, 1, 2};
    std::sort(at, at + 3, [&](int a, int b) { return r.st[a] < r.st[b]; });
    long long covered = r.d;
    for (int i : at) {
        if (r.ext[i] <= 1)
            continue;
        if (r.st[i] < covered)
            return false;
        covered += r.st[i] * (r.ext[i] - 1);
    }
    return true;
}

// Whether two row sets share no element, as far as can be told: their spans
// are apart, or they are side by side in the cells of one layout (for some
// stride C, each set is a window smaller than C repeated at multiples of C,
// and the windows of a cell are apart), as q and k in one packed projection
// output or the keys and values of one [pages][2]... cache.
bool apart(const Rows &a, const Rows &b)
{
    if (empty(a) || empty(b) ||
        !overlap(a.p, static_cast<size_t>(extent_of(a)) * 2, b.p, static_cast<size_t>(extent_of(b)) * 2))
        return true;
    const long long delta_bytes = static_cast<long long>(reinterpret_cast<uintptr_t>(b.p)) -
                                  static_cast<long long>(reinterpret_cast<uintptr_t>(a.p));
    const long long delta = delta_bytes / 2;  // bases are 16-byte aligned
    const Rows *both[2] = {&a, &b};
    for (const Rows *from : both)
        for (int i = 0; i < 3; ++i) {
            const long long cell = from->st[i];
            if (from->ext[i] <= 1)
                continue;
            long long window[2];
            bool regular = true;
            for (int t = 0; t < 2; ++t) {
                window[t] = both[t]->d;
                for (int k = 0; k < 3; ++k) {
                    if (both[t]->ext[k] <= 1)
                        continue;
                    if (both[t]->st[k] < cell)
                        window[t] += both[t]->st[k] * (both[t]->ext[k] - 1);
                    else
                        regular = regular && both[t]->st[k] % cell == 0;
                }
            }
            const long long at = ((delta % cell) + cell) % cell;
            if (regular && at >= window[0] && at + window[1] <= cell)
                return true;
        }
    return false;
}

bool same_rows(const Rows &a, const Rows &b)
{
    if (a.p != b.p)
        return false;
    for (int i = 0; i < 3; ++i)
        if (a.ext[i] != b.ext[i] || (a.ext[i] > 1 && a.st[i] != b.st[i]))
            return false;
    return true;
}

// An output against a plain buffer.
bool apart(const Rows &a, const void *p, size_t bytes)
{
    return empty(a) || p == nullptr || bytes == 0 ||
           !overlap(a.p, static_cast<size_t>(extent_of(a)) * 2, p, bytes);
}

bool head_dim_ok(int d) { return d == 64 || d == 96 || d == 128 || d == 256; }

// Rotation arguments shared by the norm and append calls.
fattn_status_t check_rope(const float *rope, int rot_dim, int max_pos, int d, int interleaved)
{
    if (interleaved != 0 && interleaved != 1)
        return FATTN_ERR_INVALID_ARG;
    if (rot_dim < 0 || rot_dim > d || rot_dim % 16 != 0)
        return FATTN_ERR_INVALID_ARG;
    if (rot_dim == 0)
        return FATTN_OK;
    if (!rope || !aligned16(rope) || max_pos < 1)
        return FATTN_ERR_INVALID_ARG;
    return FATTN_OK;
}

// A paged cache's geometry and the lists that describe its sequences.
struct Paging {
    const int *page_table, *cu_q, *kv_len;
    int B, num_pages, page_size, max_pages;
    long long table_stride;
};

fattn_status_t check_paging(const Paging &g)
{
    if (g.B < 0 || g.num_pages < 0 || g.max_pages < 0)
        return FATTN_ERR_INVALID_ARG;
    if (g.page_size < 16 || (g.page_size & (g.page_size - 1)) != 0)
        return FATTN_ERR_UNSUPPORTED;
    // Positions are 32-bit.
    if (static_cast<long long>(g.max_pages) * g.page_size > 0x7fffffffLL - 256)
        return FATTN_ERR_UNSUPPORTED;
    return FATTN_OK;
}

fattn_status_t check_lists(const Paging &g)
{
    if (!g.cu_q || !g.kv_len || (!g.page_table && g.max_pages > 0))
        return FATTN_ERR_INVALID_ARG;
    if (g.B > 1 && (g.table_stride < g.max_pages || g.table_stride > (1LL << 38)))
        return FATTN_ERR_INVALID_ARG;
    const int *lists[3] = {g.page_table, g.cu_q, g.kv_len};
    for (const int *l : lists)
        if (reinterpret_cast<uintptr_t>(l) % 4 != 0)
            return FATTN_ERR_INVALID_ARG;
    return FATTN_OK;
}

size_t table_bytes(const Paging &g)
{
    return g.B == 0 || g.max_pages == 0
               ? 0
               : static_cast<size_t>(g.table_stride * (g.B - 1) + g.max_pages) * 4;
}

// Device pointers of a call (null entries are skipped) on the current device.
template <size_t n>
fattn_status_t check_buffers(const void *const (&bufs)[n], int *dev, DeviceInfo *info)
{
    fattn_status_t s = current_device(dev, info);
    for (size_t i = 0; i < n && s == FATTN_OK; ++i)
        if (bufs[i] != nullptr)
            s = check_device_buffer(bufs[i], *dev);
    return s;
}

fattn_status_t status_word(uint32_t **out)
{
    const cudaError_t e = fattn::status_word_address(out);
    return e == cudaSuccess ? FATTN_OK : cuda_fail(e);
}

void copy_strides(long long (&dst)[3], const Rows &r)
{
    for (int i = 0; i < 3; ++i)
        dst[i] = r.st[i];
}

// Both passes of the norm and rotation.  g, dw and the workspace belong to
// the backward pass (backward true), whose outputs are y = dx.
struct NormCall {
    const void *x[2], *g[2], *w[2];
    void *y[2];
    float *dw[2];
    const long long *x_st[2], *g_st[2], *y_st[2];
};

fattn_status_t norm_rope(const NormCall &c, bool backward, const float *rope, const int *positions,
                         int B, int Hq, int Hk, int N, int d, int rot_dim, int max_pos, float eps,
                         int interleaved, int dtype, void *workspace, size_t workspace_bytes,
                         cudaStream_t stream)
{
    if (B < 0 || Hq < 0 || Hk < 0 || N < 0 || (dtype != 0 && dtype != 1))
        return FATTN_ERR_INVALID_ARG;
    if (!(eps > 0.f) || !isfinite(eps))
        return FATTN_ERR_INVALID_ARG;
    if (!head_dim_ok(d))
        return FATTN_ERR_UNSUPPORTED;
    fattn_status_t s = check_rope(rope, rot_dim, max_pos, d, interleaved);
    if (s != FATTN_OK)
        return s;
    const int H[2] = {Hq, Hk};
    const bool any_w = (Hq > 0 && c.w[0]) || (Hk > 0 && c.w[1]);
    if (backward)
        for (int t = 0; t < 2; ++t)
            if (H[t] > 0 && (c.w[t] != nullptr) != (c.dw[t] != nullptr))
                return FATTN_ERR_INVALID_ARG;
    const long long tokens = static_cast<long long>(B) * N;
    if (tokens > 0x7fffffffLL - 64)
        return FATTN_ERR_UNSUPPORTED;
    if (tokens == 0 || Hq + static_cast<long long>(Hk) == 0) {
        // No rows: the sums of an empty set are zero.
        for (int t = 0; t < 2 && backward; ++t) {
            if (H[t] == 0 || !c.dw[t])
                continue;
            int dev = 0;
            DeviceInfo info;
            const void *bufs[1] = {c.dw[t]};
            if (reinterpret_cast<uintptr_t>(c.dw[t]) % 4 != 0)
                return FATTN_ERR_INVALID_ARG;
            if ((s = check_buffers(bufs, &dev, &info)) != FATTN_OK)
                return s;
            const cudaError_t e = cudaMemsetAsync(c.dw[t], 0, static_cast<size_t>(d) * 4, stream);
            if (e != cudaSuccess)
                return cuda_fail(e);
        }
        return FATTN_OK;
    }
    // Inputs and outputs of each present tensor.
    Rows x[2] = {}, g[2] = {}, y[2] = {};
    for (int t = 0; t < 2; ++t) {
        if (H[t] == 0)
            continue;
        if (!c.y_st[t] || (backward && !c.g_st[t]))
            return FATTN_ERR_INVALID_ARG;
        const bool reads_x = !backward || c.w[t] != nullptr;
        if (reads_x && !c.x_st[t])
            return FATTN_ERR_INVALID_ARG;
        y[t] = rows_of(c.y[t], c.y_st[t], 3, B, H[t], N, d);
        if ((s = check_rows(y[t])) != FATTN_OK)
            return s;
        if (!distinct(y[t]))
            return FATTN_ERR_INVALID_ARG;
        if (reads_x) {
            x[t] = rows_of(c.x[t], c.x_st[t], 3, B, H[t], N, d);
            if ((s = check_rows(x[t])) != FATTN_OK)
                return s;
        }
        if (backward) {
            g[t] = rows_of(c.g[t], c.g_st[t], 3, B, H[t], N, d);
            if ((s = check_rows(g[t])) != FATTN_OK)
                return s;
        }
        if (c.w[t] && !aligned16(c.w[t]))
            return FATTN_ERR_INVALID_ARG;
        if (backward && c.dw[t] && reinterpret_cast<uintptr_t>(c.dw[t]) % 4 != 0)
            return FATTN_ERR_INVALID_ARG;
    }
    if (reinterpret_cast<uintptr_t>(positions) % 4 != 0)
        return FATTN_ERR_INVALID_ARG;
    const size_t need = backward && any_w ? fattn_qk_norm_rope_bwd_workspace_size(d) : 0;
    if (backward && any_w && need == 0)
        return FATTN_ERR_CUDA;
    if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need))
        return FATTN_ERR_INVALID_ARG;
    // Plain buffers of the call, and no output over any of them; an output
    // may be its own tensor's input (in place), else it is apart from every
    // row set.
    const size_t pos_bytes = positions ? static_cast<size_t>(tokens) * 4 : 0;
    const size_t rope_bytes = rot_dim ? static_cast<size_t>(max_pos) * rot_dim * 4 : 0;
    struct Plain {
        const void *p;
        size_t n;
        bool out;
    };
    const Plain plain[] = {{rot_dim ? rope : nullptr, rope_bytes, false},
                           {rot_dim ? positions : nullptr, pos_bytes, false},
                           {Hq ? c.w[0] : nullptr, static_cast<size_t>(d) * 2, false},
                           {Hk ? c.w[1] : nullptr, static_cast<size_t>(d) * 2, false},
                           {backward && Hq ? c.dw[0] : nullptr, static_cast<size_t>(d) * 4, true},
                           {backward && Hk ? c.dw[1] : nullptr, static_cast<size_t>(d) * 4, true},
                           {need ? workspace : nullptr, need, true}};
    for (int t = 0; t < 2; ++t) {
        if (H[t] == 0)
            continue;
        for (const Plain &q : plain)
            if (!apart(y[t], q.p, q.n))
                return FATTN_ERR_INVALID_ARG;
        for (int o = 0; o < 2; ++o) {
            if (H[o] == 0)
                continue;
            if (o > t && !apart(y[t], y[o]))
                return FATTN_ERR_INVALID_ARG;
            const bool reads_x = !backward || c.w[o] != nullptr;
            if (reads_x && !(o == t && same_rows(y[t], x[o])) && !apart(y[t], x[o]))
                return FATTN_ERR_INVALID_ARG;
            if (backward && !(o == t && same_rows(y[t], g[o])) && !apart(y[t], g[o]))
                return FATTN_ERR_INVALID_ARG;
            for (const Plain &q : plain)
                if (q.out && ((reads_x && !apart(x[o], q.p, q.n)) ||
                              (backward && !apart(g[o], q.p, q.n))))
                    return FATTN_ERR_INVALID_ARG;
        }
    }
    for (const Plain &a : plain)
        for (const Plain &b : plain)
            if (&a != &b && a.out && a.p && b.p && overlap(a.p, a.n, b.p, b.n))
                return FATTN_ERR_INVALID_ARG;
    int dev = 0;
    DeviceInfo info;
    const void *bufs[] = {Hq ? x[0].p : nullptr, Hk ? x[1].p : nullptr,
                          Hq && backward ? g[0].p : nullptr, Hk && backward ? g[1].p : nullptr,
                          Hq ? y[0].p : nullptr, Hk ? y[1].p : nullptr, plain[0].p, plain[1].p,
                          plain[2].p, plain[3].p, plain[4].p, plain[5].p, plain[6].p};
    if ((s = check_buffers(bufs, &dev, &info)) != FATTN_OK)
        return s;
    fattn::NormRopeArgs a = {};
    if ((s = status_word(&a.status)) != FATTN_OK)
        return s;
    for (int t = 0; t < 2; ++t) {
        a.H[t] = H[t];
        if (H[t] == 0)
            continue;
        a.x[t] = x[t].p;
        a.y[t] = c.y[t];
        a.w[t] = c.w[t];
        a.g[t] = backward ? g[t].p : nullptr;
        a.dw[t] = backward ? c.dw[t] : nullptr;
        copy_strides(a.x_st[t], x[t]);
        copy_strides(a.y_st[t], y[t]);
        copy_strides(a.g_st[t], g[t]);
    }
    a.partial = need > 0 ? static_cast<float *>(workspace) : nullptr;
    a.table = rope;
    a.positions = positions;
    a.tokens = tokens;
    a.N = N;
    a.d = d;
    a.rot = rot_dim;
    a.max_pos = max_pos;
    a.interleaved = interleaved;
    a.f16 = dtype;
    a.eps = eps;
    const cudaError_t e = fattn::launch_norm_rope(a, info.num_sms, stream);
    return e == cudaSuccess ? FATTN_OK : cuda_fail(e);
}

// ---------------------------------------------------------------- paged attention
// Workspace of a paged call: the CTAs' starts, then (256-byte aligned each)
// the partial log-sum-exps and the partial O of two slots a CTA.
struct PagedWs {
    size_t l, o, bytes;
    int slot_rows, tile_tokens;
};

PagedWs paged_ws(int Hq, int Hk, int d, int max_q, int num_sms)
{
    PagedWs w;
    const int G = Hq / Hk;
    w.tile_tokens = 128 / G;
    w.slot_rows = max_q <= w.tile_tokens ? (max_q * G + 31) / 32 * 32 : 256;
    w.l = align_up(2 * static_cast<size_t>(num_sms) * sizeof(int4), kWsAlign);
    w.o = align_up(w.l + 2ull * num_sms * w.slot_rows * 4, kWsAlign);
    w.bytes = w.o + 2ull * num_sms * w.slot_rows * d * 4;
    return w;
}

fattn_status_t check_heads(int Hq, int Hk, int d, int max_q)
{
    if (Hq < 0 || Hk < 0 || (Hq > 0 && (Hk == 0 || Hq % Hk != 0)) || max_q < 1)
        return FATTN_ERR_INVALID_ARG;
    if ((d != 64 && d != 96 && d != 128) || (Hq > 0 && Hq / Hk > 128))
        return FATTN_ERR_UNSUPPORTED;
    return FATTN_OK;
}

// 4-D tensor map of 16-bit rows of d elements, box (64, b1, b2, b3).  The
// stride of a dimension of extent 1 is not used; it only has to be valid.
fattn_status_t make_row_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap *m, const void *p,
                            int d, const long long (&ext)[3], const long long (&st)[3],
                            const unsigned (&box_rows)[3], bool f16)
{
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(d)}, strides[3];
    cuuint32_t box[4] = {64};
    const cuuint32_t elem_strides[4] = {1, 1, 1, 1};
    for (int i = 0; i < 3; ++i) {
        dims[i + 1] = static_cast<cuuint64_t>(ext[i]);
        strides[i] = static_cast<cuuint64_t>(ext[i] > 1 ? st[i] : d) * 2;
        box[i + 1] = box_rows[i];
    }
    const CUresult r = encode(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                              4, const_cast<void *>(p), dims, strides, box, elem_strides,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        t_last_cuda_error = static_cast<int>(r);
        return FATTN_ERR_CUDA;
    }
    return FATTN_OK;
}

}  // namespace

extern "C" {

fattn_status_t attn_fwd(const void *q, const void *k, const void *v, void *o, float *lse, int B,
                        int H, int N, int d, float scale, int causal, struct CUstream_st *stream)
{
    return forward(Kernel::kTcgen05, q, k, v, o, lse, B, H, N, d, scale, causal, stream);
}

fattn_status_t attn_fwd_fp16(const void *q, const void *k, const void *v, void *o, float *lse,
                             int B, int H, int N, int d, float scale, int causal,
                             struct CUstream_st *stream)
{
    return forward(Kernel::kTcgen05F16, q, k, v, o, lse, B, H, N, d, scale, causal, stream);
}

int attn_fwd_split_count(int B, int H, int N, int d, int causal)
{
    bool empty = false;
    if (check_shape(B, H, N, d, 1.0f, causal, &empty) != FATTN_OK)
        return 0;
    if (empty)
        return 1;
    int dev = 0;
    DeviceInfo info;
    if (current_device(&dev, &info) != FATTN_OK)
        return 0;
    return choose_splits(B, H, N, N, d, info.num_sms);
}

size_t attn_fwd_split_workspace_size(int B, int H, int N, int d, int num_splits)
{
    bool empty = false;
    if (num_splits < 1 || num_splits > kMaxSplits ||
        check_shape(B, H, N, d, 1.0f, 0, &empty) != FATTN_OK || empty)
        return 0;
    return split_ws_bytes(B, H, N, d, num_splits);
}

fattn_status_t attn_fwd_split(const void *q, const void *k, const void *v, void *o, float *lse,
                              int B, int H, int N, int d, float scale, int causal, int num_splits,
                              void *workspace, size_t workspace_bytes, struct CUstream_st *stream)
{
    if (num_splits < 1)
        return FATTN_ERR_INVALID_ARG;
    return forward_split(q, k, v, o, lse, B, H, N, N, d, scale, causal, num_splits, workspace,
                         workspace_bytes, stream);
}

fattn_status_t attn_fwd_strided(const void *q, const void *k, const void *v, void *o,
                                float *lse, int B, int H, int Nq, int Nk, int d,
                                const long long *q_strides, const long long *k_strides,
                                const long long *v_strides, const long long *o_strides,
                                float scale, int causal, int num_splits, void *workspace,
                                size_t workspace_bytes, int dtype, struct CUstream_st *stream)
{
    if (!q_strides || !k_strides || !v_strides || !o_strides || dtype < 0 || dtype > 2)
        return FATTN_ERR_INVALID_ARG;
    Layout L;
    for (int i = 0; i < 3; ++i) {
        L.q[i] = q_strides[i];
        L.k[i] = k_strides[i];
        L.v[i] = v_strides[i];
        L.o[i] = o_strides[i];
    }
    // A dimension of extent 1 has no meaningful stride: give it the span of
    // the smaller dimensions, as a contiguous tensor would have.
    long long *all[4] = {L.q, L.k, L.v, L.o};
    const int rows[4] = {Nq, Nk, Nk, Nq};
    for (int t = 0; t < 4; ++t) {
        if (rows[t] == 1)
            all[t][2] = (static_cast<long long>(d) + 7) / 8 * 8;
        if (H == 1)
            all[t][1] = all[t][2] * (rows[t] > 0 ? rows[t] : 1);
        if (B == 1)
            all[t][0] = all[t][1] * (H > 0 ? H : 1);
    }
    return forward_split(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, num_splits, workspace,
                         workspace_bytes, stream, &L,
                         dtype == 1 ? Kernel::kTcgen05F16
                                    : (dtype == 2 ? Kernel::kTcgen05Bf16P : Kernel::kTcgen05));
}

size_t attn_fwd_kv_workspace_size(int B, int H, int Nq, int Nk, int d, int causal,
                                  int num_splits)
{
    bool empty = false;
    if (num_splits < 0 || num_splits > kMaxSplits ||
        check_shape(B, H, Nq, d, 1.0f, causal, &empty) != FATTN_OK ||
        check_keys(B, H, Nq, Nk, d, causal) != FATTN_OK || empty)
        return 0;
    if (num_splits == 0) {
        int dev = 0, streamk = 0;
        DeviceInfo info;
        if (current_device(&dev, &info) != FATTN_OK)
            return 0;
        num_splits = auto_slots(B, H, Nq, Nk, d, causal, info.num_sms, &streamk);
    }
    return split_ws_bytes(B, H, Nq, d, num_splits);
}

fattn_status_t attn_fwd_kv(const void *q, const void *k, const void *v, void *o, float *lse,
                           int B, int H, int Nq, int Nk, int d, float scale, int causal,
                           int num_splits, void *workspace, size_t workspace_bytes,
                           struct CUstream_st *stream)
{
    return forward_split(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, num_splits, workspace,
                         workspace_bytes, stream);
}

fattn_status_t attn_fwd_split_noalloc(const void *q, const void *k, const void *v, void *o,
                                      float *lse, int B, int H, int N, int d, float scale,
                                      int causal, int num_splits, struct CUstream_st *stream)
{
    if (num_splits < 1 || num_splits > kMaxSplits)
        return FATTN_ERR_INVALID_ARG;
    bool empty = false;
    fattn_status_t s = check_shape(B, H, N, d, scale, causal, &empty);
    if (s != FATTN_OK || empty)
        return s;
    if (num_splits == 1)  // no scratch needed: attn_fwd's result (V converted on chip)
        return forward(Kernel::kTcgen05, q, k, v, o, lse, B, H, N, d, scale, causal, stream,
                       false);
    if (split_ws_bytes(B, H, N, d, num_splits) > kNoAllocScratchBytes)
        return FATTN_ERR_UNSUPPORTED;  // beyond the fixed scratch: use attn_fwd_split
    int dev = 0;
    DeviceInfo info;
    if ((s = current_device(&dev, &info)) != FATTN_OK)
        return s;
    void *scratch = nullptr;
    if ((s = noalloc_scratch(dev, &scratch)) != FATTN_OK)
        return s;
    return forward_split(q, k, v, o, lse, B, H, N, N, d, scale, causal, num_splits, scratch,
                         kNoAllocScratchBytes, stream, nullptr, Kernel::kTcgen05, false);
}

int fattn_set_v_conversion(int mode)
{
    if (mode < FATTN_V_CONVERT_AUTO || mode > FATTN_V_CONVERT_PREPASS)
        return -1;
    return g_v_convert.exchange(mode);
}

int fattn_v_conversion_route(int N, int d, int causal)
{
    if (N < 0 || (d != 64 && d != 96 && d != 128 && d != 256) || (causal != 0 && causal != 1))
        return -1;
    return v_route(N, d, causal) == VRoute::kPrepass ? FATTN_V_CONVERT_PREPASS
                                                     : FATTN_V_CONVERT_ON_CHIP;
}

fattn_status_t fattn_trim_scratch(void)
{
    std::lock_guard<std::mutex> lock(g_pool_mutex);
    for (int dev = 0; dev < kMaxDevices; ++dev) {
        if (g_pool[dev] == nullptr)
            continue;
        const cudaError_t e = cudaMemPoolTrimTo(g_pool[dev], 0);
        if (e != cudaSuccess)
            return cuda_fail(e);
    }
    return FATTN_OK;
}

size_t attn_bwd_workspace_size(int B, int H, int N, int d)
{
    bool empty = false;
    if ((d != 64 && d != 128) || check_shape(B, H, N, d, 1.0f, 0, &empty) != FATTN_OK || empty)
        return 0;
    return static_cast<size_t>(B) * H * N * sizeof(float);
}

fattn_status_t attn_bwd(const void *q, const void *k, const void *v, const void *o,
                        const float *lse, const void *dout, void *dq, void *dk, void *dv, int B,
                        int H, int N, int d, float scale, int causal, void *workspace,
                        size_t workspace_bytes, struct CUstream_st *stream)
{
    bool empty = false;
    fattn_status_t s = check_shape(B, H, N, d, scale, causal, &empty);
    if (s != FATTN_OK || empty)
        return s;
    if (d != 64 && d != 128)  // the backward kernels take d = 64 or 128
        return FATTN_ERR_UNSUPPORTED;
    const size_t rows = static_cast<size_t>(B) * H * N;
    const size_t tb = rows * d * 2, lb = rows * 4;
    const void *ins[6] = {q, k, v, o, lse, dout};
    const size_t in_bytes[6] = {tb, tb, tb, tb, lb, tb};
    void *outs[4] = {dq, dk, dv, workspace};
    const size_t out_bytes[4] = {tb, tb, tb, lb};
    for (const void *p : ins)
        if (!p || !aligned16(p))
            return FATTN_ERR_INVALID_ARG;
    for (void *p : outs)
        if (!p || !aligned16(p))
            return FATTN_ERR_INVALID_ARG;
    if (workspace_bytes < lb)
        return FATTN_ERR_INVALID_ARG;
    // Outputs (and the scratch) overlap neither each other nor any input.
    for (int a = 0; a < 4; ++a) {
        for (int i = 0; i < 6; ++i)
            if (overlap(outs[a], out_bytes[a], ins[i], in_bytes[i]))
                return FATTN_ERR_INVALID_ARG;
        for (int c = a + 1; c < 4; ++c)
            if (overlap(outs[a], out_bytes[a], outs[c], out_bytes[c]))
                return FATTN_ERR_INVALID_ARG;
    }
    int dev = 0;
    DeviceInfo info;
    if ((s = current_device(&dev, &info)) != FATTN_OK)
        return s;
    for (const void *p : ins)
        if ((s = check_device_buffer(p, dev)) != FATTN_OK)
            return s;
    for (void *p : outs)
        if ((s = check_device_buffer(p, dev)) != FATTN_OK)
            return s;
    PFN_cuTensorMapEncodeTiled_v12000 encode;
    if ((s = get_encoder(&encode)) != FATTN_OK)
        return s;
    fattn::FwdMaps maps;
    fattn::BwdMaps bmaps;
    const long long BH = static_cast<long long>(B) * H;
    if ((s = make_map(encode, &maps.q, q, N, d, BH)) != FATTN_OK ||
        (s = make_map(encode, &maps.k, k, N, d, BH)) != FATTN_OK ||
        (s = make_map(encode, &maps.v, v, N, d, BH)) != FATTN_OK ||
        (s = make_map(encode, &bmaps.dout, dout, N, d, BH)) != FATTN_OK)
        return s;
    uint32_t *status = nullptr;
    cudaError_t e = fattn::status_word_address(&status);
    if (e != cudaSuccess)
        return cuda_fail(e);
    fattn::BwdArgs a{q, k, v, o, dout, lse, dq, dk, dv, static_cast<float *>(workspace), status,
                     B, H, N, d, scale, causal};
    e = fattn::launch_bwd_sm103(a, maps, bmaps, info.num_sms, stream);
    return e == cudaSuccess ? FATTN_OK : cuda_fail(e);
}

static fattn_status_t rowop(bool softmax, const void *x, void *y, int M, int N, int dtype,
                            cudaStream_t stream)
{
    if (M < 0 || N < 0 || (dtype != 0 && dtype != 1))
        return FATTN_ERR_INVALID_ARG;
    if (M == 0 || (N == 0 && softmax))
        return FATTN_OK;
    if (!y || (!x && N > 0))
        return FATTN_ERR_INVALID_ARG;
    if (N == 0) {  // row sums of empty rows are zero; x is not read
        if (reinterpret_cast<uintptr_t>(y) % 4)
            return FATTN_ERR_INVALID_ARG;
        int dev = 0;
        DeviceInfo info;
        fattn_status_t s = current_device(&dev, &info);
        if (s != FATTN_OK || (s = check_device_buffer(y, dev)) != FATTN_OK)
            return s;
        const cudaError_t e = cudaMemsetAsync(y, 0, static_cast<size_t>(M) * 4, stream);
        return e == cudaSuccess ? FATTN_OK : cuda_fail(e);
    }
    const size_t elem = dtype == 0 ? 4 : 2;
    const size_t in_bytes = static_cast<size_t>(M) * N * elem;
    const size_t out_bytes = softmax ? in_bytes : static_cast<size_t>(M) * 4;
    if (reinterpret_cast<uintptr_t>(x) % elem || reinterpret_cast<uintptr_t>(y) % 4 ||
        (softmax && reinterpret_cast<uintptr_t>(y) % elem))
        return FATTN_ERR_INVALID_ARG;
    // The softmax may run in place (y == x) but not on partly overlapping
    // buffers; the row sums must not overlap the input.
    if ((!softmax || x != y) && overlap(x, in_bytes, y, out_bytes))
        return FATTN_ERR_INVALID_ARG;
    int dev = 0;
    DeviceInfo info;
    fattn_status_t s = current_device(&dev, &info);
    if (s != FATTN_OK)
        return s;
    if ((s = check_device_buffer(x, dev)) != FATTN_OK || (s = check_device_buffer(y, dev)) != FATTN_OK)
        return s;
    const cudaError_t e =
        softmax ? fattn::launch_softmax_rows(x, y, M, N, dtype, info.num_sms, stream)
                : fattn::launch_row_sum(x, static_cast<float *>(y), M, N, dtype, info.num_sms, stream);
    return e == cudaSuccess ? FATTN_OK : cuda_fail(e);
}

fattn_status_t fattn_softmax_rows(const void *x, void *y, int M, int N, int dtype,
                                  struct CUstream_st *stream)
{
    return rowop(true, x, y, M, N, dtype, stream);
}

fattn_status_t fattn_row_sum(const void *x, float *out, int M, int N, int dtype,
                             struct CUstream_st *stream)
{
    return rowop(false, x, out, M, N, dtype, stream);
}

fattn_status_t attn_fwd_simt(const void *q, const void *k, const void *v, void *o, float *lse,
                             int B, int H, int N, int d, float scale, int causal,
                             struct CUstream_st *stream)
{
    return forward(Kernel::kSimt, q, k, v, o, lse, B, H, N, d, scale, causal, stream);
}

fattn_status_t attn_fwd_host(const void *q_host, const void *k_host, const void *v_host,
                             void *o_host, float *lse_host, void *dq, void *dk, void *dv, void *do_,
                             float *dlse, int B, int H, int N, int d, float scale, int causal,
                             struct CUstream_st *stream)
{
    bool empty = false;
    int dev = 0;
    DeviceInfo info;
    fattn_status_t s = validate(dq, dk, dv, do_, dlse, B, H, N, N, d, scale, causal, &empty, &dev,
                                &info);
    if (s != FATTN_OK || empty)
        return s;
    if (!q_host || !k_host || !v_host || !o_host || !lse_host)
        return FATTN_ERR_INVALID_ARG;
    // Heads are independent, so the copies and the compute are pipelined
    // over chunks of consecutive (b, h) heads: copies in on one helper
    // stream, the kernel on `stream`, copies out on another, ordered by
    // events.  The helper streams first wait for the work already on
    // `stream`; the call returns after everything has completed.
    std::lock_guard<std::mutex> lock(g_pipe_mutex);
    HostPipe *hp = nullptr;
    if ((s = host_pipe(dev, &hp)) != FATTN_OK)
        return s;
    const long long BH = static_cast<long long>(B) * H;
    long long bounds[kHostChunks + 1];
    const long long q_tiles = (static_cast<long long>(N) + 127) / 128;
    const long long units = d == 256 ? q_tiles : (q_tiles + 1) / 2;  // work units per head
    const int chunks = host_chunk_plan(BH, (info.num_sms + units - 1) / units, bounds);
    const size_t head_bytes = static_cast<size_t>(N) * d * 2, head_lse = static_cast<size_t>(N) * 4;
    auto at = [](const void *base, size_t off) {
        return static_cast<const uint8_t *>(base) + off;
    };
    auto atw = [](void *base, size_t off) { return static_cast<uint8_t *>(base) + off; };
    cudaError_t e = cudaEventRecord(hp->start, stream);
    if (e == cudaSuccess)
        e = cudaStreamWaitEvent(hp->in, hp->start, 0);
    if (e == cudaSuccess)
        e = cudaStreamWaitEvent(hp->out, hp->start, 0);
    for (int c = 0; c < chunks && e == cudaSuccess && s == FATTN_OK; ++c) {
        const long long h0 = bounds[c], h1 = bounds[c + 1];
        const size_t off = static_cast<size_t>(h0) * head_bytes;
        const size_t bytes = static_cast<size_t>(h1 - h0) * head_bytes;
        if ((e = cudaMemcpyAsync(atw(dq, off), at(q_host, off), bytes, cudaMemcpyHostToDevice,
                                 hp->in)) != cudaSuccess ||
            (e = cudaMemcpyAsync(atw(dk, off), at(k_host, off), bytes, cudaMemcpyHostToDevice,
                                 hp->in)) != cudaSuccess ||
            (e = cudaMemcpyAsync(atw(dv, off), at(v_host, off), bytes, cudaMemcpyHostToDevice,
                                 hp->in)) != cudaSuccess ||
            (e = cudaEventRecord(hp->ev_in[c], hp->in)) != cudaSuccess ||
            (e = cudaStreamWaitEvent(stream, hp->ev_in[c], 0)) != cudaSuccess)
            break;
        float *lse_c = reinterpret_cast<float *>(atw(dlse, static_cast<size_t>(h0) * head_lse));
        if ((s = launch(Kernel::kTcgen05, info, at(dq, off), at(dk, off), at(dv, off),
                        atw(do_, off), lse_c, 1, static_cast<int>(h1 - h0), N, N, d, scale, causal,
                        stream)) != FATTN_OK)
            break;
        if ((e = cudaEventRecord(hp->ev_done[c], stream)) != cudaSuccess ||
            (e = cudaStreamWaitEvent(hp->out, hp->ev_done[c], 0)) != cudaSuccess ||
            (e = cudaMemcpyAsync(atw(o_host, off), at(do_, off), bytes, cudaMemcpyDeviceToHost,
                                 hp->out)) != cudaSuccess ||
            (e = cudaMemcpyAsync(atw(lse_host, static_cast<size_t>(h0) * head_lse), lse_c,
                                 static_cast<size_t>(h1 - h0) * head_lse, cudaMemcpyDeviceToHost,
                                 hp->out)) != cudaSuccess)
            break;
    }
    // Drain all three streams whatever happened, so that no copy still
    // touches the caller's buffers after the return.
    const cudaError_t e_in = cudaStreamSynchronize(hp->in);
    const cudaError_t e_st = cudaStreamSynchronize(stream);
    const cudaError_t e_out = cudaStreamSynchronize(hp->out);
    if (s != FATTN_OK)
        return s;
    for (cudaError_t x : {e, e_in, e_st, e_out})
        if (x != cudaSuccess)
            return cuda_fail(x);
    return FATTN_OK;
}

fattn_status_t fattn_qk_norm_rope(const void *q, const void *k, void *q_out, void *k_out,
                                  const void *wq, const void *wk, const float *rope,
                                  const int *positions, int B, int Hq, int Hk, int N, int d,
                                  int rot_dim, int max_pos, const long long *q_strides,
                                  const long long *k_strides, const long long *q_out_strides,
                                  const long long *k_out_strides, float eps, int interleaved,
                                  int dtype, struct CUstream_st *stream)
{
    NormCall c = {};
    c.x[0] = q;
    c.x[1] = k;
    c.y[0] = q_out;
    c.y[1] = k_out;
    c.w[0] = wq;
    c.w[1] = wk;
    c.x_st[0] = q_strides;
    c.x_st[1] = k_strides;
    c.y_st[0] = q_out_strides;
    c.y_st[1] = k_out_strides;
    return norm_rope(c, false, rope, positions, B, Hq, Hk, N, d, rot_dim, max_pos, eps, interleaved,
                     dtype, nullptr, 0, stream);
}

size_t fattn_qk_norm_rope_bwd_workspace_size(int d)
{
    int dev = 0;
    DeviceInfo info;
    if (!head_dim_ok(d) || current_device(&dev, &info) != FATTN_OK)
        return 0;
    return static_cast<size_t>(fattn::norm_rope_bwd_blocks(info.num_sms)) * d * 4;
}

fattn_status_t fattn_qk_norm_rope_bwd(const void *dq_out, const void *dk_out, const void *q,
                                      const void *k, const void *wq, const void *wk,
                                      const float *rope, const int *positions, void *dq, void *dk,
                                      float *dwq, float *dwk, int B, int Hq, int Hk, int N, int d,
                                      int rot_dim, int max_pos, const long long *dq_out_strides,
                                      const long long *dk_out_strides, const long long *q_strides,
                                      const long long *k_strides, const long long *dq_strides,
                                      const long long *dk_strides, float eps, int interleaved,
                                      int dtype, void *workspace, size_t workspace_bytes,
                                      struct CUstream_st *stream)
{
    NormCall c = {};
    c.x[0] = q;
    c.x[1] = k;
    c.g[0] = dq_out;
    c.g[1] = dk_out;
    c.y[0] = dq;
    c.y[1] = dk;
    c.w[0] = wq;
    c.w[1] = wk;
    c.dw[0] = dwq;
    c.dw[1] = dwk;
    c.x_st[0] = q_strides;
    c.x_st[1] = k_strides;
    c.g_st[0] = dq_out_strides;
    c.g_st[1] = dk_out_strides;
    c.y_st[0] = dq_strides;
    c.y_st[1] = dk_strides;
    return norm_rope(c, true, rope, positions, B, Hq, Hk, N, d, rot_dim, max_pos, eps, interleaved,
                     dtype, workspace, workspace_bytes, stream);
}

fattn_status_t fattn_kv_append(const void *k, const void *v, void *k_cache, void *v_cache,
                               const int *page_table, const int *cu_q, const int *kv_len,
                               const float *rope, int T, int B, int Hk, int d, int num_pages,
                               int page_size, int max_pages, long long page_table_stride,
                               int rot_dim, int max_pos, const long long *k_strides,
                               const long long *v_strides, const long long *k_cache_strides,
                               const long long *v_cache_strides, int interleaved, int dtype,
                               struct CUstream_st *stream)
{
    if (T < 0 || Hk < 0 || (dtype != 0 && dtype != 1))
        return FATTN_ERR_INVALID_ARG;
    if (!head_dim_ok(d))
        return FATTN_ERR_UNSUPPORTED;
    const Paging g{page_table, cu_q, kv_len, B, num_pages, page_size, max_pages, page_table_stride};
    fattn_status_t s = check_paging(g);
    if (s != FATTN_OK || (s = check_rope(rope, rot_dim, max_pos, d, interleaved)) != FATTN_OK)
        return s;
    if (T == 0 || B == 0 || Hk == 0)
        return FATTN_OK;
    if ((s = check_lists(g)) != FATTN_OK)
        return s;
    if (!k_strides || !v_strides || !k_cache_strides || !v_cache_strides || num_pages == 0)
        return FATTN_ERR_INVALID_ARG;
    const Rows in[2] = {rows_of(k, k_strides, 2, T, Hk, 1, d), rows_of(v, v_strides, 2, T, Hk, 1, d)};
    const Rows out[2] = {rows_of(k_cache, k_cache_strides, 3, num_pages, Hk, page_size, d),
                         rows_of(v_cache, v_cache_strides, 3, num_pages, Hk, page_size, d)};
    const size_t lists[4] = {table_bytes(g), (static_cast<size_t>(B) + 1) * 4,
                             static_cast<size_t>(B) * 4,
                             rot_dim ? static_cast<size_t>(max_pos) * rot_dim * 4 : 0};
    const void *list[4] = {page_table, cu_q, kv_len, rope};
    for (const Rows &r : in)
        if ((s = check_rows(r)) != FATTN_OK)
            return s;
    for (const Rows &r : out) {
        if ((s = check_rows(r)) != FATTN_OK)
            return s;
        if (!distinct(r) || !apart(r, in[0]) || !apart(r, in[1]))
            return FATTN_ERR_INVALID_ARG;
        for (int i = 0; i < 4; ++i)
            if (lists[i] > 0 && !apart(r, list[i], lists[i]))
                return FATTN_ERR_INVALID_ARG;
    }
    if (!apart(out[0], out[1]))
        return FATTN_ERR_INVALID_ARG;
    int dev = 0;
    DeviceInfo info;
    const void *bufs[] = {k, v, k_cache, v_cache, max_pages ? page_table : nullptr, cu_q, kv_len,
                          rot_dim ? rope : nullptr};
    if ((s = check_buffers(bufs, &dev, &info)) != FATTN_OK)
        return s;
    fattn::KvAppendArgs a = {};
    if ((s = status_word(&a.status)) != FATTN_OK)
        return s;
    a.k = k;
    a.v = v;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.page_table = page_table;
    a.cu_q = cu_q;
    a.kv_len = kv_len;
    a.table = rope;
    for (int i = 0; i < 2; ++i) {
        a.k_st[i] = in[0].st[i];
        a.v_st[i] = in[1].st[i];
    }
    copy_strides(a.kc_st, out[0]);
    copy_strides(a.vc_st, out[1]);
    a.table_stride = page_table_stride;
    a.T = T;
    a.B = B;
    a.H = Hk;
    a.d = d;
    a.rot = rot_dim;
    a.max_pos = max_pos;
    a.interleaved = interleaved;
    a.f16 = dtype;
    a.num_pages = num_pages;
    a.page_shift = __builtin_ctz(static_cast<unsigned>(page_size));
    a.max_pages = max_pages;
    const cudaError_t e = fattn::launch_kv_append(a, info.num_sms, stream);
    return e == cudaSuccess ? FATTN_OK : cuda_fail(e);
}

size_t attn_fwd_paged_workspace_size(int Hq, int Hk, int d, int max_q)
{
    int dev = 0;
    DeviceInfo info;
    if (Hq == 0 || check_heads(Hq, Hk, d, max_q) != FATTN_OK || current_device(&dev, &info) != FATTN_OK)
        return 0;
    return paged_ws(Hq, Hk, d, max_q, info.num_sms).bytes;
}

fattn_status_t attn_fwd_paged(const void *q, const void *k_cache, const void *v_cache,
                              const int *page_table, const int *cu_q, const int *kv_len, void *o,
                              float *lse, int T, int B, int Hq, int Hk, int d, int num_pages,
                              int page_size, int max_pages, long long page_table_stride, int max_q,
                              const long long *q_strides, const long long *k_cache_strides,
                              const long long *v_cache_strides, const long long *o_strides,
                              float scale, int causal, int dtype, void *workspace,
                              size_t workspace_bytes, struct CUstream_st *stream)
{
    if (T < 0 || (dtype != 0 && dtype != 1) || (causal != 0 && causal != 1))
        return FATTN_ERR_INVALID_ARG;
    if (T > 0x7fffffff - 256)  // token indexes are 32-bit, tiles included
        return FATTN_ERR_UNSUPPORTED;
    if (!(scale > 0.f) || !isfinite(scale))
        return FATTN_ERR_INVALID_ARG;
    const Paging g{page_table, cu_q, kv_len, B, num_pages, page_size, max_pages, page_table_stride};
    fattn_status_t s = check_heads(Hq, Hk, d, max_q);
    if (s != FATTN_OK || (s = check_paging(g)) != FATTN_OK)
        return s;
    if (T == 0 || B == 0 || Hq == 0)
        return FATTN_OK;
    if ((s = check_lists(g)) != FATTN_OK)
        return s;
    if (!q_strides || !k_cache_strides || !v_cache_strides || !o_strides || num_pages == 0 || !lse ||
        reinterpret_cast<uintptr_t>(lse) % 4 != 0)
        return FATTN_ERR_INVALID_ARG;
    const Rows rows[4] = {rows_of(q, q_strides, 2, T, Hq, 1, d),
                          rows_of(k_cache, k_cache_strides, 3, num_pages, Hk, page_size, d),
                          rows_of(v_cache, v_cache_strides, 3, num_pages, Hk, page_size, d),
                          rows_of(o, o_strides, 2, T, Hq, 1, d)};
    for (const Rows &r : rows)
        if ((s = check_rows(r)) != FATTN_OK)
            return s;
    // The tensor map steps from one key head's query heads to the next's.
    if (Hq > 1 && rows[0].st[1] > (1LL << 38) / (Hq / Hk))
        return FATTN_ERR_UNSUPPORTED;
    const Rows &out = rows[3];
    const size_t lse_bytes = static_cast<size_t>(T) * Hq * 4;
    const size_t lists[3] = {table_bytes(g), (static_cast<size_t>(B) + 1) * 4, static_cast<size_t>(B) * 4};
    const void *list[3] = {page_table, cu_q, kv_len};
    if (!distinct(out) || !apart(out, lse, lse_bytes))
        return FATTN_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)
        if (!apart(out, rows[i]) || !apart(rows[i], lse, lse_bytes) || !apart(out, list[i], lists[i]) ||
            (lists[i] > 0 && overlap(lse, lse_bytes, list[i], lists[i])))
            return FATTN_ERR_INVALID_ARG;
    int dev = 0;
    DeviceInfo info;
    const void *bufs[] = {q, k_cache, v_cache, o, lse, max_pages ? page_table : nullptr, cu_q, kv_len,
                          workspace};
    if ((s = check_buffers(bufs, &dev, &info)) != FATTN_OK)
        return s;
    const PagedWs ws = paged_ws(Hq, Hk, d, max_q, info.num_sms);
    if (!workspace || !aligned16(workspace) || workspace_bytes < ws.bytes ||
        overlap(workspace, ws.bytes, lse, lse_bytes))
        return FATTN_ERR_INVALID_ARG;
    for (int i = 0; i < 4; ++i)
        if (!apart(rows[i], workspace, ws.bytes) ||
            (i < 3 && lists[i] > 0 && overlap(workspace, ws.bytes, list[i], lists[i])))
            return FATTN_ERR_INVALID_ARG;
    PFN_cuTensorMapEncodeTiled_v12000 encode;
    if ((s = get_encoder(&encode)) != FATTN_OK)
        return s;
    fattn::PagedArgs a = {};
    if ((s = status_word(&a.status)) != FATTN_OK)
        return s;
    const int G = Hq / Hk;
    const int box_tokens = std::min(max_q, ws.tile_tokens), quad_tokens = std::min(max_q, 32 / G);
    const unsigned box_slots = static_cast<unsigned>(page_size < 128 ? page_size : 128);
    fattn::PagedMaps maps;
    const long long q_ext[3] = {G, Hk, T}, q_st[3] = {rows[0].st[1], rows[0].st[1] * G, rows[0].st[0]};
    if ((s = make_row_map(encode, &maps.q, q, d, q_ext, q_st,
                          {static_cast<unsigned>(G), 1u, static_cast<unsigned>(box_tokens)},
                          dtype == 1)) != FATTN_OK)
        return s;
    maps.q_quad = maps.q;
    if (quad_tokens > 0 && quad_tokens != box_tokens &&
        (s = make_row_map(encode, &maps.q_quad, q, d, q_ext, q_st,
                          {static_cast<unsigned>(G), 1u, static_cast<unsigned>(quad_tokens)},
                          dtype == 1)) != FATTN_OK)
        return s;
    CUtensorMap *cache[2] = {&maps.k, &maps.v};
    for (int i = 0; i < 2; ++i) {
        const Rows &r = rows[1 + i];
        if ((s = make_row_map(encode, cache[i], r.p, d, {page_size, Hk, num_pages},
                              {r.st[2], r.st[1], r.st[0]}, {box_slots, 1u, 1u}, dtype == 1)) != FATTN_OK)
            return s;
    }
    uint8_t *base = static_cast<uint8_t *>(workspace);
    a.o = o;
    a.lse = lse;
    a.starts = reinterpret_cast<int4 *>(base);
    a.ws_l = reinterpret_cast<float *>(base + ws.l);
    a.ws_o = reinterpret_cast<float *>(base + ws.o);
    a.page_table = page_table;
    a.cu_q = cu_q;
    a.kv_len = kv_len;
    a.o_st[0] = out.st[0];
    a.o_st[1] = out.st[1];
    a.table_stride = page_table_stride;
    a.T = T;
    a.B = B;
    a.Hk = Hk;
    a.G = G;
    a.d = d;
    a.f16 = dtype;
    a.causal = causal;
    a.max_q = max_q;
    a.num_pages = num_pages;
    a.page_shift = __builtin_ctz(static_cast<unsigned>(page_size));
    a.max_keys = max_pages * page_size;
    a.tile_tokens = ws.tile_tokens;
    a.q_box_tokens = box_tokens;
    a.q_quad_tokens = quad_tokens;
    a.slot_rows = ws.slot_rows;
    a.g_inverse = (65536u + G - 1) / G;
    a.sl2 = scale * 1.4426950408889634f;
    const cudaError_t e = fattn::launch_paged(a, maps, info.num_sms, stream);
    return e == cudaSuccess ? FATTN_OK : cuda_fail(e);
}

const char *fattn_status_string(fattn_status_t status)
{
    switch (status) {
    case FATTN_OK: return "FATTN_OK";
    case FATTN_ERR_INVALID_ARG: return "FATTN_ERR_INVALID_ARG";
    case FATTN_ERR_UNSUPPORTED: return "FATTN_ERR_UNSUPPORTED";
    case FATTN_ERR_CUDA: return "FATTN_ERR_CUDA";
    case FATTN_ERR_TIMEOUT: return "FATTN_ERR_TIMEOUT";
    case FATTN_ERR_RANGE: return "FATTN_ERR_RANGE";
    case FATTN_ERR_INDEX: return "FATTN_ERR_INDEX";
    }
    return "FATTN_UNKNOWN_STATUS";
}

int fattn_last_cuda_error(void) { return t_last_cuda_error; }

fattn_status_t fattn_get_device_status(int *status, struct CUstream_st *stream)
{
    if (!status)
        return FATTN_ERR_INVALID_ARG;
    uint32_t word = 0;
    const cudaError_t e = fattn::read_and_clear_status(&word, stream);
    if (e != cudaSuccess)
        return cuda_fail(e);
    *status = static_cast<int>(word);
    if (word == 0)
        return FATTN_OK;
    const uint32_t code = word & 0xffu;
    return code == FATTN_ERR_RANGE   ? FATTN_ERR_RANGE
           : code == FATTN_ERR_INDEX ? FATTN_ERR_INDEX
                                     : FATTN_ERR_TIMEOUT;
}

fattn_status_t fattn_selftest_wait_timeout(unsigned int limit_us, struct CUstream_st *stream)
{
    if (limit_us == 0 || limit_us > 2000000u)
        return FATTN_ERR_INVALID_ARG;
    int dev = 0;
    DeviceInfo info;
    fattn_status_t s = current_device(&dev, &info);
    if (s != FATTN_OK)
        return s;
    const cudaError_t e =
        fattn::launch_selftest_wait_timeout(static_cast<uint64_t>(limit_us) * 1000u, stream);
    return e == cudaSuccess ? FATTN_OK : cuda_fail(e);
}

const char *fattn_version(void) { return "libfattn 0.1.0 sm_103a"; }

}  // extern "C"
