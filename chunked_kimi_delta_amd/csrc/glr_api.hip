// glr_api.hip -- the extern "C" boundary of the gated linear recurrence (include/glr.h): argument
// checks, workspace layout and the launches on the caller's stream. Host side only.
#include <math.h>

#include "glr_scan.h"

namespace kda {
int current_device_cus();
}

namespace {

using namespace glr;

constexpr int64_t MOST = 1 << 18;       // channels, and elements from one token to the next

bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
size_t align256(size_t x) { return (x + 255) / 256 * 256; }

kda_status check_shapes(const glr_args *a)
{
    if (!a) return KDA_ERR_INVALID_ARG;
    if (a->B < 1 || a->T < 0 || a->N < 1 || a->D < 1) return KDA_ERR_INVALID_ARG;
    if (a->cu_seqlens) {
        if (a->B != 1 || !aligned(a->cu_seqlens, 8)) return KDA_ERR_INVALID_ARG;
    } else if (a->N != a->B) {
        return KDA_ERR_INVALID_ARG;
    }
    if (a->io != KDA_BF16 && a->io != KDA_FP32) return KDA_ERR_UNSUPPORTED;
    if (a->D > MOST) return KDA_ERR_UNSUPPORTED;
    if (a->gate != KDA_GATE_NONE && a->gate != KDA_GATE_SOFTPLUS && a->gate != KDA_GATE_BOUNDED)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status check_tensors(const glr_args *a, bool x_read)
{
    const uintptr_t e = a->io == KDA_FP32 ? 4 : 2;
    if ((int64_t)a->B * a->T > 0) {
        if ((x_read && !a->x) || !a->g || !a->y) return KDA_ERR_INVALID_ARG;
        if (!aligned(a->x, e) || !aligned(a->g, e) || !aligned(a->beta, e) || !aligned(a->y, e)) return KDA_ERR_INVALID_ARG;
        const int64_t strides[] = {x_read ? a->x_stride : a->D, a->g_stride, a->beta ? a->beta_stride : a->D};
        const int64_t batches[] = {x_read ? a->x_batch : 0, a->g_batch, a->beta ? a->beta_batch : 0};
        for (int i = 0; i < 3; ++i) {
            if (strides[i] < a->D) return KDA_ERR_INVALID_ARG;
            if (strides[i] > MOST) return KDA_ERR_UNSUPPORTED;
            if (a->B > 1 && batches[i] != 0 && batches[i] < (a->T - 1) * strides[i] + a->D) return KDA_ERR_INVALID_ARG;
        }
    }
    if (!aligned(a->initial_state, 4) || !aligned(a->final_state, 4)) return KDA_ERR_INVALID_ARG;
    if (a->gate == KDA_GATE_NONE) return KDA_OK;
    if (!a->A_log || !aligned(a->A_log, 4) || !aligned(a->dt_bias, 4)) return KDA_ERR_INVALID_ARG;
    if (a->gate == KDA_GATE_BOUNDED && !(a->gate_lower_bound < 0.f && a->gate_lower_bound > -INFINITY))
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

// Two channels a lane where every row begins at a multiple of two elements.
int vec_of(const glr_args *a, bool x_read, const void *const *more, int n)
{
    const uintptr_t e = a->io == KDA_FP32 ? 8 : 4;
    auto even = [&](const void *p, int64_t stride, int64_t batch) {
        return aligned(p, e) && stride % 2 == 0 && (a->B == 1 || batch % 2 == 0);
    };
    bool two = a->D % 2 == 0 && even(a->g, a->g_stride, a->g_batch) && aligned(a->y, e);
    if (x_read) two = two && even(a->x, a->x_stride, a->x_batch);
    if (a->beta) two = two && even(a->beta, a->beta_stride, a->beta_batch);
    for (int i = 0; i < n; ++i) two = two && aligned(more[i], e);
    return two ? 2 : 1;
}

// Tiles that hand states to each other, or strips of whole sequences? Strips are one launch and no workspace (13 us a
// call, tiles 18), and the better of the two wherever strips of 64 channels fill the device; narrower ones take longer, and
// a packed batch's longest sequence takes its time alone. bf16, us, strips and tiles: 4 x 4096 tokens x 4096 channels 86 and 98
// (gradients 147 and 149, raw 247 and 273); 2560 x 4096 21 and 24 (28 and 27, raw 73 and 60), 3300 x 4096 24 and 29 (51 and 36, raw 92
// and 76), 7000 x 4096 68 and 50; 3300 x 2048 19 and 19 (28 and 23), 16384 x 1000 83 and 38. One switch for the forward and the
// gradients, so near it one of them is a fifth from its better side (forward of 3300 x 4096, gradients of 3300 x 2048).
// Packed, 16 x 2048 tokens x 4096 183 and 185, 7 x 512 + 16384 x 2048 125 and 66, 32 x 512 x 2048 37 and 45 (gradients 73 and 79, raw
// 121 and 145). Lengths lie on the device, and the mean stands for them: a batch of one long sequence among many short ones
// takes strips and the long one's time, 8000 + 31 x 100 x 2048 141 and 42 (gradients 240 and 54, raw 430 and 115), 32768 + 63 x 1
// x 2048 564 and 118.
bool use_tiles(const glr_args *a)
{
    const int64_t tokens = (int64_t)a->B * a->T, mean = tokens / a->N;
    const int64_t channels = (int64_t)a->N * a->D, cus = kda::current_device_cus();
    if (a->cu_seqlens && a->N > 1) return mean >= 1024 && tokens >= 8192;
    return channels < 64 * cus && mean >= (channels < 16 * cus ? 3584 : 2560);
}

// Tiles have 64 lanes a token, and one channel a lane where two would take the registers of a second workgroup on a
// compute unit (fp32 gradients 102 -> 71 us for 8192 x 2048, bf16 with beta 280 -> 250 for 4 x 8192 x 4096; without, 373 against 407
// for 131072 x 2048; bf16 gradients 324 -> 281 for 4 x 8192 x 4096, with beta 155 against 161 for 4 x 4096 x 2048).
// Strips have as many lanes a token as leave every compute unit a workgroup: 8 x 1000 tokens x 2048 channels, raw, 38 us with
// 64, 41, 52 and 68 with 32, 16 and 8; 2048 x 2048 13 us with 8 and 40 with 64.
Shape shape_of(const glr_args *a, int vec, bool back)
{
    const bool f32 = a->io == KDA_FP32;
    if (use_tiles(a)) return Shape{f32, true, !f32 && back == (a->beta != nullptr) ? vec : 1, 64};
    int lanes = 64;
    while (lanes > 8 && (int64_t)a->N * ((a->D + lanes - 1) / lanes) < kda::current_device_cus()) lanes /= 2;
    return Shape{f32, false, 1, lanes};
}

Params params_of(const glr_args *a, Shape s)
{
    Params p = {};
    p.seq.cu = a->cu_seqlens;
    p.seq.T = a->T;
    p.seq.T_total = (int64_t)a->B * a->T;
    p.seq.N = a->N;
    p.D = a->D;
    p.strips = (a->D + s.vec * s.lanes - 1) / (s.vec * s.lanes);
    p.x = a->x;
    p.g = a->g;
    p.beta = a->beta;
    p.xs = a->x_stride;
    p.gs = a->g_stride;
    p.bs = a->beta_stride;
    auto beyond = [&](int64_t batch, int64_t stride) { return a->B > 1 && batch != 0 ? batch - a->T * stride : 0; };
    p.xe = beyond(a->x_batch, a->x_stride);
    p.ge = beyond(a->g_batch, a->g_stride);
    p.be = beyond(a->beta_batch, a->beta_stride);
    p.h0 = a->initial_state;
    p.y = a->y;
    p.ht = a->final_state;
    p.pre = Pre{a->beta_sigmoid != 0, a->gate, a->gate_lower_bound, a->A_log, a->dt_bias};
    return p;
}

// A launch has less than 2^32 threads.
bool fits(const glr_args *a, Shape s)
{
    const int ch = s.vec * s.lanes;
    const int64_t strips = (a->D + ch - 1) / ch, most = ((int64_t)1 << 32) - 1;
    if (s.tiles)                // of at least 64 tokens, workgroups of at most 512 threads
        return (((int64_t)a->B * a->T) / 64 + a->N) * strips <= most / 512;
    return unit_grid(strips, a->N, near_of(ch * (s.f32 ? 4 : 2))) <= most / (64 * W);
}

// Workspace of the tiles for either number of channels a lane (alignments are not known yet).
size_t tiles_workspace(const glr_args *a, bool back)
{
    int64_t most = 0;
    for (int vec = 1; vec <= 2; ++vec) {
        const Shape s = {a->io == KDA_FP32, true, vec, 64};
        const Params p = params_of(a, s);
        const int64_t n = back ? tiles_back_bytes(p, s) : tiles_bytes(p, s);
        most = n > most ? n : most;
    }
    return align256((size_t)most);
}

}  // namespace

extern "C" {

size_t glr_fwd_workspace_bytes(const glr_args *a)
{
    return check_shapes(a) == KDA_OK && use_tiles(a) ? tiles_workspace(a, false) : 0;
}

kda_status glr_fwd(const glr_args *a, void *workspace, size_t ws_bytes, void *stream)
{
    kda_status st = check_shapes(a);
    if (st != KDA_OK || (st = check_tensors(a, true)) != KDA_OK) return st;
    const Shape s = shape_of(a, vec_of(a, true, nullptr, 0), false);
    if (!fits(a, s)) return KDA_ERR_UNSUPPORTED;
    const size_t need = glr_fwd_workspace_bytes(a);
    if (need && (!workspace || ws_bytes < need || !aligned(workspace, 256))) return KDA_ERR_WORKSPACE;
    const Params p = params_of(a, s);
    hipStream_t hs = (hipStream_t)stream;
    return (s.tiles ? launch_fwd_tiles(p, s, workspace, hs) : launch_fwd(p, s, hs)) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t glr_bwd_workspace_bytes(const glr_args *a)
{
    if (check_shapes(a) != KDA_OK) return 0;
    const bool tiles = use_tiles(a);
    const int64_t rows = tiles ? tiles_back_rows(params_of(a, Shape{a->io == KDA_FP32, true, 1, 64})) : a->N;
    return (a->gate ? 2 * align256((size_t)rows * a->D * 4) : 0) + (tiles ? tiles_workspace(a, true) : 0);
}

kda_status glr_bwd(const glr_args *a, const void *d_y, const float *dht, void *workspace, size_t ws_bytes,
                   void *dx, void *dg, void *dbeta, float *dh0, float *dA_log, float *ddt_bias, void *stream)
{
    kda_status st = check_shapes(a);
    if (st != KDA_OK || (st = check_tensors(a, a->beta != nullptr)) != KDA_OK) return st;
    const uintptr_t e = a->io == KDA_FP32 ? 4 : 2;
    const bool gated = a->gate != KDA_GATE_NONE;
    const void *io[] = {d_y, dx, dg, a->beta ? dbeta : dg};
    if ((int64_t)a->B * a->T > 0)
        for (const void *p : io)
            if (!p || !aligned(p, e)) return KDA_ERR_INVALID_ARG;
    if (!aligned(dht, 4) || !aligned(dh0, 4)) return KDA_ERR_INVALID_ARG;
    if (gated && (!dA_log || !aligned(dA_log, 4) || !aligned(ddt_bias, 4))) return KDA_ERR_INVALID_ARG;
    const Shape s = shape_of(a, vec_of(a, a->beta != nullptr, io, 4), true);
    if (!fits(a, s)) return KDA_ERR_UNSUPPORTED;
    const size_t need = glr_bwd_workspace_bytes(a);
    if (need && (!workspace || ws_bytes < need || !aligned(workspace, 256))) return KDA_ERR_WORKSPACE;
    BwdParams q = {};
    q.f = params_of(a, s);
    q.d_y = d_y;
    q.dht = dht;
    q.dx = dx;
    q.dg = dg;
    q.dbeta = dbeta;
    q.dh0 = dh0;
    const bool tiles = s.tiles;
    const int64_t rows = tiles ? tiles_back_rows(q.f) : a->N;
    const size_t part = gated ? align256((size_t)rows * a->D * 4) : 0;
    uint8_t *const ws = (uint8_t *)workspace;
    q.part_A = (float *)ws;
    q.part_b = (float *)(ws + part);
    hipStream_t hs = (hipStream_t)stream;
    if ((tiles ? launch_bwd_tiles(q, s, ws + 2 * part, hs) : launch_bwd(q, s, hs)) != hipSuccess) return KDA_ERR_HIP;
    if (gated && launch_params(q, rows, dA_log, ddt_bias, hs) != hipSuccess) return KDA_ERR_HIP;
    return KDA_OK;
}

kda_status glr_step(const glr_args *a, float *state, const int32_t *state_indices, int32_t slots, void *stream)
{
    kda_status st = check_shapes(a);
    if (st != KDA_OK) return st;
    if (a->cu_seqlens || slots < 0 || (!state_indices && slots < a->B)) return KDA_ERR_INVALID_ARG;
    if ((st = check_tensors(a, true)) != KDA_OK) return st;
    if (a->T == 0) return KDA_OK;
    if ((slots > 0 && !state) || !aligned(state, 4) || !aligned(state_indices, 4)) return KDA_ERR_INVALID_ARG;
    const int vec = vec_of(a, true, nullptr, 0);
    StepParams p = {};
    p.f = params_of(a, Shape{a->io == KDA_FP32, false, vec, 1});
    p.state = state;
    p.index = state_indices;
    p.B = a->B;
    p.T = a->T;
    p.slots = slots;
    if ((int64_t)a->B * p.f.strips >= ((int64_t)1 << 32) - 256) return KDA_ERR_UNSUPPORTED;
    return launch_step(p, a->io == KDA_FP32, vec, (hipStream_t)stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
