// Internal interface between the C ABI (api.cpp) and the gfx950 kernels.
// Everything here is launched on the caller's stream; nothing synchronises.
#pragma once

#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

namespace ifx {

// Arguments of one implicit-GEMM convolution launch.
struct ConvArgs {
    const int8_t *x;       // packed input  [n, i1, h, w, 32]
    const int8_t *wt;      // packed weights [o1, kh, kw, i1, o2, 32]
    const int32_t *bias;   // [oc]
    const int32_t *mult;   // [oc]
    const int32_t *shift;  // [oc]
    const int8_t *res;     // packed shortcut [n, oc1, ho, wo, 32] or null
    void *y;               // packed int8 output, or int32 NHWC when out_i32
    int n, h, w, i1;       // input batch, size, channel blocks
    int ho, wo, oc, oc1;   // output size, channels, channel blocks
    int o2;                // output-channel group of the weight layout
    int stride, pad;
    int m;                 // n * ho * wo (GEMM rows)
    int nkb;               // kh * kw * i1 (32-wide reduction blocks)
    int relu, residual, out_i32;
    int out_even;          // store only the even rows and columns of the output (chained conv3)
    // or null: also store the even rows and columns of the output, densely, here
    // ([n, oc1, ceil(ho / 2), ceil(wo / 2), 32]): the input of a following stride-2 projection
    int8_t *y_even;
    // phase-split layout [n][c1][2][2][h/2][w/2][32] (even sizes): plane (y % 2, x % 2) holds the
    // pixels of that row and column parity, so a stride-2 3x3 reads contiguous runs for every tap
    int in_ps, out_ps;
    // split-K (partial launches only): workgroup row blockIdx.y covers 32-channel blocks
    // [blockIdx.y * kb_per, +kb_per) of the reduction and writes its int32 sums, without the
    // bias, to slice blockIdx.y of y ([ksplit][m][oc]); ksplit = 1 is the whole reduction
    int ksplit, kb_per;
    // magic numbers for exact unsigned division of n < 2^31 by ho*wo, wo, o2
    // (q = n when d == 1, else umulhi(n, mul) >> shr); see fastdiv_magic()
    unsigned howo_mul, wo_mul, o2_mul;
    int howo_shr, wo_shr, o2_shr;
};

// Host-side kernel-name query.  While a thread has a query armed, the launchers it reaches
// launch nothing: the first one writes the name of the kernel instance it would launch, as
// profilers print it (e.g. "igemm_kernel<3, 3, 128, 128, 2, false, true, false>"), and returns
// hipSuccess.  The query therefore runs exactly the dispatch code of the launch it describes.
struct KernelQuery {
    char name[160];
    bool answered;
    bool even_copy;  // the answering launcher writes ConvArgs::y_even
};
KernelQuery *&armed_query();  // this thread's armed query, or null

// Called first by every leaf launcher: true when a query took the call (nothing to launch).
// even_copy: the launcher writes ConvArgs::y_even.
inline bool answer_query_e(bool even_copy, const char *fmt, va_list ap)
{
    KernelQuery *q = armed_query();
    if (!q) return false;
    if (!q->answered) {
        vsnprintf(q->name, sizeof(q->name), fmt, ap);
        q->answered = true;
        q->even_copy = even_copy;
    }
    return true;
}
inline bool answer_query_even(bool even_copy, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    const bool r = answer_query_e(even_copy, fmt, ap);
    va_end(ap);
    return r;
}
inline bool answer_query(const char *fmt, ...)
{
    KernelQuery *q = armed_query();
    if (!q) return false;
    if (!q->answered) {
        va_list ap;
        va_start(ap, fmt);
        vsnprintf(q->name, sizeof(q->name), fmt, ap);
        va_end(ap);
        q->answered = true;
        q->even_copy = false;
    }
    return true;
}

inline const char *tf(bool b) { return b ? "true" : "false"; }

// Compute units of the current device: a device property the runtime keeps on the host, so
// reading it launches nothing and is safe while a stream is being captured.  The persistent
// kernels size their grids from it and from their compile-time residency per CU.
inline hipError_t current_cus(int *cus)
{
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipSuccess) e = hipDeviceGetAttribute(cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e == hipSuccess && *cus < 1) *cus = 1;
    return e;
}

// The compute units a rule may count on, asked of the runtime once a thread and device (256 without one).
inline int cus_or_default()
{
    thread_local int known_dev = -1, known = 256;
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess) return 256;
    if (dev != known_dev) {
        if (current_cus(&cus) != hipSuccess) return 256;
        known = cus;
        known_dev = dev;
    }
    return known;
}

// Magic multiplier and shift for q = floor(n / d), 0 <= n < 2^31, d >= 1:
// with p = 31 + ceil(log2 d) and m = ceil(2^p / d), floor(n * m / 2^p) = floor(n / d)
// (the classic round-up method for dividing by an invariant integer; m < 2^32).
inline void fastdiv_magic(unsigned d, unsigned *mul, int *shr)
{
    if (d <= 1) {
        *mul = 0;
        *shr = 0;
        return;
    }
    int l = 0;
    while ((1ull << l) < d) ++l;
    const int p = 31 + l;
    *mul = (unsigned)(((1ull << p) + d - 1) / d);
    *shr = p - 32;
}

// Arguments of the fused stem (7x7/s2/p3 conv + ReLU + 3x3/s2/p1 max-pool).
struct StemArgs {
    const int8_t *x;       // packed input [n, 1, h, w, 32], or compact NHWC [n, h, w, c] when nhwc
    const int8_t *wt;      // stem weights [oc=64, 8, 8, 4]
    const int32_t *bias, *mult, *shift;
    int8_t *y;             // packed pooled output [n, 2, ph, pw, 32]
    int n, h, w, c;        // input (c <= 4)
    int nhwc;              // input layout: 0 packed, 1 compact NHWC
    int ho, wo;            // conv output
    int ph, pw;            // pooled output
    int relu;
};

// Inputs of the BN folding kernel (device pointers; see ifx_fold_bn).
struct FoldArgs {
    int c_out;
    float x_scale, y_scale, eps;
    int w_per_channel;
    const float *w_scale, *conv_bias, *gamma, *beta, *mean, *var;
};

// One product of two microscaled 4-bit tensors (device pointers; see ifx_mx4_matmul).
struct Mx4Args {
    const uint8_t *a_codes, *a_scales;  // [k1][m][64], [k1][m][4]
    const uint8_t *w_codes, *w_scales;  // [k1][n][64], [k1][n][4]
    const float *bias;                  // [n] or null
    const void *res;                    // rows of n every ld_res elements, of `type`, or null
    void *y;                            // rows of n every ld_y elements, of `type`
    int m, n, k1;
    int type, act;
    long long ld_y, ld_res;
    int past;  // set by the launcher: y is stored past the caches (stored_past)
};

// One product of two 8-bit tensors, or the gated pair of projections and its gradient (device pointers; see
// ifx_fp8_matmul, ifx_gated, ifx_gated_fp8 and ifx_gated_backward).
struct Fp8Args {
    const uint8_t *a_codes, *a_scales;  // [k1][m][128], [ceil(k1 / 4)][m][4]
    const uint8_t *w_codes, *w_scales;  // [k1][n][128], [ceil(k1 / 4)][n][4]: the weights, or the gate's
    const uint8_t *u_codes, *u_scales;  // the other projection's (gated forms)
    const float *bias;                  // [n] or null (product)
    const void *res;                    // residual or null (product), dy (gradient), of `type`
    void *y, *y2;                       // result, of `type`; of the gradient: at the gate and at the other projection
    uint8_t *codes, *scales;            // instead of y: 8-bit codes of n columns (gated form; else null)
    float *ws;                          // [m][n]: its values for few rows
    int m, n, k1;
    int a_format, type, act;
    long long ld_y, ld_y2, ld_res;
    int past;  // set by the launcher: y is stored past the caches (stored_past)
};

// One root mean square norm or its gradient (device pointers; see ifx_rms_norm).
struct RmsArgs {
    const void *x, *res;      // forward: input, residual or null
    const void *dy, *dh;      // gradient: of the norm, past the norm (or null)
    void *h, *y;              // forward: the sum (or null), the norm (null in the 8-bit form); gradient: x is the sum, y is dx
    uint8_t *codes, *scales;  // forward: instead of y (else null)
    const float *weight;      // [c] or null
    float *rstd;              // [rows]; written by the forward pass (or null), read by the gradient
    float *part;              // gradient: partial sums of dweight, [chunks][c] (null: no dweight)
    int rows, c, type;
    float eps;
    long long ld_x, ld_res, ld_h, ld_y, ld_dy, ld_dh;
    int past, chunks;  // set by the launcher
};

// Whether rows of a result are stored past the caches: they begin on 128-byte lines, so that stores fill whole
// lines, and there are more bytes than would stay in the L2s (4 MB in each of eight) until they are read.
// us, cached / past: product 100352 x 128 x 512 14.9 / 11.8, 50176 x 512 x 128 17.2 / 15.5, 4096^3 39.8 / 37.7;
// 4-bit values of 200704 x 512 48 / 38, but of 100000 rows of 1000 bf16, which share lines, 62 / 74; a
// group norm's split form, 4 x 12544 x 1024 forward 70 / 58, its gradient 120 / 110, of 128 x 3136 x 256 228 / 208
// (its one-read forms were slower past the caches, 51 / 54 for 128 x 784 x 512, and keep to them).
inline bool stored_past(const void *y, long long rows, long long ld, int bytes)
{
    return ld * bytes % 128 == 0 && (reinterpret_cast<uintptr_t>(y) & 127u) == 0 && rows * ld * bytes > (16 << 20);
}

// One group norm or its gradient (device pointers; see ifx_group_norm).
struct GnArgs {
    const void *x, *dy;
    void *y;                     // y, or dx of the gradient
    uint8_t *codes, *scales;     // instead of y: microscaled 4-bit codes (else null)
    const float *weight, *bias;  // [c] or null
    float *mean, *rstd;          // [n][groups]; written by the forward pass (or null), read by the gradient
    float *ws, *gsum;
    int n, hw, c, groups;
    int type, act;
    float eps;
    long long ld_x, ld_dy, ld_y;
    // set by the launcher: results stored past the caches (stored_past), channels of a group and their
    // division, lanes that sum one group, chunks of a sample and their pixels
    int past;
    int cg, cg_shr;
    unsigned cg_mul;
    int lpg, chunks, px;
    // the resident form: groups of a span, spans of a sample, (sample, span) pairs of an XCD,
    // division by cg / 8
    int gs, spans, per_xcd;
    unsigned cgv_mul;
    int cgv_shr;
};

hipError_t launch_conv(const ConvArgs &a, int kh, int kw, hipStream_t s);
// Whether the kernel launch_conv_split picks for `a` honours a.in_ps / a.out_ps (the general
// kernel does; a launch it would split over K is not given a phase-split output).
bool conv_phase_supported(const ConvArgs &a, int kh, int kw);
// Bytes of int32 partial sums launch_conv_split would use for `a` (0: it would not split).  A
// convolution on few output tiles with a long reduction is split over workgroups along K.
size_t splitk_bytes(const ConvArgs &a, int kh, int kw);
// launch_conv, split along K when that pays and `part` (part_bytes of device memory) holds the
// partial sums; a second kernel then sums them and applies the epilogue.  Results are identical.
hipError_t launch_conv_split(const ConvArgs &a, int kh, int kw, int32_t *part, size_t part_bytes, hipStream_t s);
// The 1x1 shortcut conv `a` (RESIDUAL) of a bottleneck fused with its 1x1 projection shortcut
// `pj` (same output pixels and channels, no ReLU): the projection's requantised output is the
// shortcut and never reaches HBM; a.res is not read.
hipError_t launch_conv_proj(const ConvArgs &a, const ConvArgs &pj, hipStream_t s);
// input quantisation (fp32 or uint8 NHWC image -> int8 codes) and logits dequantisation, quant.hip
hipError_t launch_quantize(const void *x, bool u8, int8_t *q, int count, int c, const float *mean, const float *mult,
                           hipStream_t s);
hipError_t launch_dequantize(const int32_t *q, float *y, int count, float scale, hipStream_t s);
// microscaled 4-bit rounding and product, mx4.hip
hipError_t launch_mx4_quantize(const void *x, int type, long long ld, int rows, int k, uint8_t *codes, uint8_t *scales,
                               hipStream_t s);
hipError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int rows, int k, void *y, int type,
                                 long long ld, hipStream_t s);
hipError_t launch_mx4_matmul(const Mx4Args &a, hipStream_t s);
hipError_t launch_mx4_tiles(Mx4Args a, hipStream_t s);  // its tiled form, mx4_gemm.hip
// 8-bit rounding, values and products, fp8.hip; the tiled forms, fp8_gemm.hip and fp8_gated.hip
hipError_t launch_fp8_quantize(const void *x, int type, long long ld, int rows, int k, int format, uint8_t *codes,
                               uint8_t *scales, hipStream_t s);
hipError_t launch_fp8_quantize_t(const void *x, int type, long long ld, int rows, int k, int format, uint8_t *codes,
                                 uint8_t *scales, hipStream_t s);
hipError_t launch_fp8_dequantize(const uint8_t *codes, const uint8_t *scales, int format, int rows, int k, void *y,
                                 int type, long long ld, hipStream_t s);
enum Fp8Mode { kProduct, kGated, kGatedGrad };
// Whether a launch of these sizes takes the few-rows form (whose 8-bit results pass through Fp8Args::ws).
bool fp8_few_rows(int m, int n);
hipError_t launch_fp8(Fp8Args a, Fp8Mode mode, hipStream_t s);
hipError_t launch_fp8_product(Fp8Args a, hipStream_t s);
hipError_t launch_fp8_gated(Fp8Args a, Fp8Mode mode, hipStream_t s);
// root mean square norm and its gradient, rms.hip
size_t rms_workspace_bytes(int rows, int c, int type);
hipError_t launch_rms_norm(RmsArgs a, hipStream_t s);
hipError_t launch_rms_norm_grad(RmsArgs a, float *dweight, hipStream_t s);
// group norm with an activation and its gradient, norm.hip
bool gn_supported(int n, int hw, int c, int groups);
size_t gn_workspace_bytes(int n, int hw, int c, int groups, int type, bool grad, bool mx4);
hipError_t launch_group_norm(GnArgs a, hipStream_t s);
hipError_t launch_group_norm_grad(GnArgs a, float *dweight, float *dbias, hipStream_t s);
hipError_t launch_fold_bn(const FoldArgs &f, int32_t *bias, int32_t *mult, int32_t *shift, int32_t *status,
                          hipStream_t s);
// 1x1 convolutions with at most 128 input channels (conv1x1.hip)
bool conv1x1_small_k_supported(const ConvArgs &a, int kh, int kw);
bool conv1x1_proj_supported(const ConvArgs &a, const ConvArgs &pj);
bool conv1x1_ring_proj_supported(const ConvArgs &a, const ConvArgs &pj);
bool conv1x1_ring_wide_supported(const ConvArgs &a);
hipError_t launch_conv1x1_ring_wide(const ConvArgs &a, hipStream_t s);
hipError_t launch_conv1x1_ring_proj(const ConvArgs &a, const ConvArgs &pj, hipStream_t s);
hipError_t launch_conv1x1_proj(const ConvArgs &a, const ConvArgs &pj, hipStream_t s);
hipError_t launch_conv1x1_small_k(const ConvArgs &a, hipStream_t s);
// conv3 of one bottleneck (a, with its shortcut) chained with conv1 of the next (b): the block
// output a.y is stored and conv1 reads it from LDS (conv1x1.hip)
bool conv1x1_chain_supported(const ConvArgs &a, const ConvArgs &b);
hipError_t launch_conv1x1_chain(const ConvArgs &a, const ConvArgs &b, hipStream_t s);
bool conv1x1_proj_chain_supported(const ConvArgs &a, const ConvArgs &pj, const ConvArgs &b);
hipError_t launch_conv1x1_proj_chain(const ConvArgs &a, const ConvArgs &pj, const ConvArgs &b, hipStream_t s);
hipError_t launch_stem(const StemArgs &a, hipStream_t s);
hipError_t launch_avgpool(const int8_t *x, int8_t *y, int n, int c1, int hw, hipStream_t s);
hipError_t launch_pack_act(const int8_t *x, int8_t *blk, int n, int h, int w, int c, hipStream_t s);
hipError_t launch_unpack_act(const int8_t *blk, int8_t *x, int n, int h, int w, int c, hipStream_t s);
hipError_t launch_pack_weights(const int8_t *w, int8_t *blk, int oc, int kh, int kw, int ic, int o2,
                               hipStream_t s);
hipError_t launch_pack_weights_stem(const int8_t *w, int8_t *blk, int oc, int ic, hipStream_t s);

}  // namespace ifx
