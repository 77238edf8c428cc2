// gdn_api.hip -- the extern "C" boundary of the gated delta rule (include/gdn.h): argument
// checks, workspace layout and the launches on the caller's stream. Host side only.
#include <math.h>

#include "gdn.h"
#include "gdn_internal.h"

namespace {

using namespace gdn;

bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
size_t align256(size_t x) { return (x + 255) / 256 * 256; }

kda_status check_shapes(const gdn_args *a)
{
    if (!a) return KDA_ERR_INVALID_ARG;
    if (a->B < 1 || a->T < 0 || a->N < 0 || a->H < 1 || a->HV < 1 || a->HV % a->H)
        return KDA_ERR_INVALID_ARG;
    if (a->cu_seqlens) {
        if (a->B != 1 || a->N < 1) return KDA_ERR_INVALID_ARG;
    } else if (a->N != a->B) {
        return KDA_ERR_INVALID_ARG;
    }
    if ((a->K != 64 && a->K != 128) || (a->V != 64 && a->V != 128)) return KDA_ERR_UNSUPPORTED;
    if (a->io != KDA_BF16 && a->io != KDA_FP32) return KDA_ERR_UNSUPPORTED;
    // grid sizes, and 32-bit offsets inside the 64 rows of a chunk
    const int64_t tt = (int64_t)a->B * a->T;
    if (a->HV > 32768 || (int64_t)a->N * a->HV > INT32_MAX || tt / CT + a->N > INT32_MAX)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status check_pre(const gdn_args *a)
{
    if (a->gate != KDA_GATE_NONE && a->gate != KDA_GATE_SOFTPLUS && a->gate != KDA_GATE_BOUNDED)
        return KDA_ERR_UNSUPPORTED;
    if (a->gate == KDA_GATE_NONE) return KDA_OK;
    if (!a->A_log || !aligned(a->A_log, 4) || !aligned(a->dt_bias, 4)) return KDA_ERR_INVALID_ARG;
    if (a->gate == KDA_GATE_BOUNDED &&
        !(a->gate_lower_bound < 0.f && a->gate_lower_bound > -INFINITY))
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

Pre pre_of(const gdn_args *a)
{
    return Pre{a->qk_l2norm != 0, a->beta_sigmoid != 0, a->gate, a->gate_lower_bound, a->A_log,
               a->dt_bias};
}

float scale_of(const gdn_args *a)
{
    return a->scale > 0.f && !isnan(a->scale) ? a->scale : 1.0f / sqrtf((float)a->K);
}

// What the chunked kernels take: a launch has less than 2^32 threads along a dimension (up to 1024 a chunk or a
// pair of sequence and value head, fp32 io: 32 a row of q or k that is split).
kda_status check_chunks(const gdn_args *a)
{
    const kda_status st = check_shapes(a);
    if (st != KDA_OK) return st;
    const int64_t tt = (int64_t)a->B * a->T;
    if (tt / CT + a->N >= 1 << 22 || (int64_t)a->N * a->HV >= (1 << 21) - 8) return KDA_ERR_UNSUPPORTED;
    return a->io == KDA_FP32 && tt * a->HV >= 1 << 26 ? KDA_ERR_UNSUPPORTED : KDA_OK;
}

// A dense batch of short sequences takes the recurrence: a chunk has a fixed cost of 64 tokens.
bool recurrent(const gdn_args *a) { return !a->cu_seqlens && a->T <= 16; }

// What a chunk takes, us, by kernel: a workgroup of the whole-sequence pass alone, of the last pass over
// segments with every compute unit busy, and of the first pass (bf16 io: two workgroups a compute unit; fp32 io:
// its three planes leave LDS for one, and counting two understates that pass. Counted in rounds of one, fp32
// forwards took 84 -> 80 us for 2 x 1000 tokens of 8 heads, 124 -> 110 for 4096 of 4, 217 -> 193 for 16384 of 2,
// but 148 -> 163 for 8192 of 8 at K = 64, whose chunks cost less than these times say: kept as it is).
struct ChunkTimes {
    double whole, last, first;
};

// The number of segments with the shortest expected time, from the number of (sequence, value head) units
// and the mean length (the lengths of packed sequences lie on the device). Joining takes 2.1 us a segment,
// two more launches about 6 us. The first pass's workgroups share compute units two by two and take 15% longer
// once a third waits. Measured, 16 heads x 4096, bf16 io, state pass of the forward: whole 206 us; 4 segments
// 97, 6: 87, 8: 77, 11: 103, 16: 97 us. Whole backward in segments of 32 chunks 374 us, 16: 262, 11: 224, 8:
// 216, 4: 234, 2: 284; 8 heads x 16384: 32: 532, 16: 422, 8: 441 (calls repeated on one set of inputs; 229 for 216
// with inputs that change). 8 packed sequences x 32 heads: whole 465 us,
// two or more segments 660 us and up (512 workgroups fill the device already).
//
// Packed sequences that would go whole, and leave no compute unit two workgroups, are cut at one and a half
// times the mean length: even batches hardly notice, a long sequence no longer sets the time alone. Forward
// (backward) us, 16 heads, K = V = 128: 8 x 2048 tokens 194 -> 202 (637 -> 641), 7 x 512 + 16384 tokens 867 ->
// 452 (1946 -> 1177), 3 .. 8192 tokens 482 -> 469 (1262 -> 1228). The last with 32 heads 586 -> 768 (1750 ->
// 2064): there the last pass fills the device either way, and the first one only adds to it.
Segments plan_segments(int64_t tt, int64_t N, bool packed, int64_t HV, int K, int ends_parts, int last_parts,
                       ChunkTimes us)
{
    Segments g = {};
    if (tt == 0) return g;
    const int64_t n = (tt / N + CT - 1) / CT, units = N * HV, cus = kda::current_device_cus();
    auto rounds = [](int64_t x, int64_t y) { return (double)((x + y - 1) / y); };
    double best = 0.95 * rounds(units * last_parts, cus) * n * us.whole;
    for (int64_t count = 2; count <= 64; ++count) {
        const int64_t len = (n + count - 1) / count;
        if (len < 2) break;
        const double first = (double)(units * ((count - 1) * ends_parts + (count - 2) * (K / 64))) / (2 * cus);
        const double t = (first > 1.0 ? 1.15 * first : 1.0) * len * us.first + (count - 2) * 2.1 + 6.0 +
                         rounds(units * count * last_parts, cus) * len * us.last;
        if (t < best) {
            best = t;
            g.chunks = (int32_t)len;
        }
    }
    if (g.chunks == 0 && packed && N > 1 && n >= 16 && units * last_parts <= cus)
        g.chunks = (int32_t)(n + n / 2);
    if (g.chunks) g.slots = (int32_t)(tt / (CT * (int64_t)g.chunks) + N);
    return g;
}

struct Layout {                     // byte offsets in the workspace
    int64_t tt, slots;
    size_t q, k, total;             // three bf16 planes each of q and k (fp32 io)
    Segments seg;
    size_t E, PHI;
};

Layout layout(const gdn_args *a)
{
    Layout L = {};
    L.tt = (int64_t)a->B * a->T;
    L.slots = L.tt / CT + a->N;
    const bool f32 = a->io == KDA_FP32;
    L.q = (size_t)L.slots * a->HV * (f32 ? Rec<3>::BYTES : Rec<2>::BYTES);
    const size_t planes = f32 ? align256((size_t)L.tt * a->H * a->K * 6) : 0;
    L.k = L.q + planes;
    L.E = L.k + planes;
    L.seg = plan_segments(L.tt, a->N, a->cu_seqlens != nullptr, a->HV, a->K, a->V / 64, a->V / 64,
                          f32 ? ChunkTimes{7.8, 8.7, 5.2} : ChunkTimes{3.2, 4.1, 3.8});
    const size_t ends = (size_t)L.seg.slots * a->HV * a->K * 4;
    L.PHI = L.E + ends * a->V;
    L.total = L.PHI + 2 * ends * a->K;
    return L;
}

template <class F>
hipError_t by_dims(int K, int V, F f)
{
    using std::integral_constant;
    if (K == 64)
        return V == 64 ? f(integral_constant<int, 64>(), integral_constant<int, 64>())
                       : f(integral_constant<int, 64>(), integral_constant<int, 128>());
    return V == 64 ? f(integral_constant<int, 128>(), integral_constant<int, 64>())
                   : f(integral_constant<int, 128>(), integral_constant<int, 128>());
}

kda_status run_recurrent(const gdn_args *a, const float *h0, float *ht, const int32_t *index,
                         int32_t slots, hipStream_t st)
{
    // rows are the grid's second dimension
    StepParams p = {};
    p.T = a->T;
    p.H = a->H;
    p.HV = a->HV;
    p.G = a->HV / a->H;
    p.scale = scale_of(a);
    p.pre = pre_of(a);
    const int64_t e = a->io == KDA_FP32 ? 4 : 2;
    for (int b = 0; b < a->N; b += 65535) {
        const int64_t tok = (int64_t)b * a->T, state = (int64_t)b * a->HV * a->K * a->V;
        p.B = a->N - b < 65535 ? a->N - b : 65535;
        p.q = (const uint8_t *)a->q + tok * a->H * a->K * e;
        p.k = (const uint8_t *)a->k + tok * a->H * a->K * e;
        p.v = (const uint8_t *)a->v + tok * a->HV * a->V * e;
        p.g = (const uint8_t *)a->g + tok * a->HV * e;
        p.beta = (const uint8_t *)a->beta + tok * a->HV * e;
        p.o = (uint8_t *)a->o + tok * a->HV * a->V * e;
        p.index = index ? index + b : nullptr;
        p.h0 = h0 && !index ? h0 + state : h0;
        p.ht = ht && !index ? ht + state : ht;
        p.slots = index ? slots : p.B;
        const hipError_t er = by_dims(a->K, a->V, [&](auto k, auto v) {
            return launch_recurrent<decltype(k)::value, decltype(v)::value>(p, a->io == KDA_FP32, st);
        });
        if (er != hipSuccess) return KDA_ERR_HIP;
    }
    return KDA_OK;
}

kda_status check_tensors(const gdn_args *a)
{
    const void *ptrs[] = {a->q, a->k, a->v, a->g, a->beta, a->o};
    if ((int64_t)a->B * a->T > 0)
        for (const void *p : ptrs)
            if (!p || !aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    const void *opt[] = {a->initial_state, a->final_state, a->cu_seqlens};
    for (const void *p : opt)
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    return check_pre(a);
}

// The fields of the forward and the backward that do not depend on the workspace.
Params params_of(const gdn_args *a, const Layout &L)
{
    Params p = {};
    p.seq.cu = a->cu_seqlens;
    p.seq.T = a->T;
    p.seq.T_total = L.tt;
    p.seq.N = a->N;
    p.seq.n_slots = (int32_t)L.slots;
    p.H = a->H;
    p.HV = a->HV;
    p.G = a->HV / a->H;
    p.scale = scale_of(a);
    p.q[0] = (const uint16_t *)a->q;
    p.k[0] = (const uint16_t *)a->k;
    p.v = a->v;
    p.g = a->g;
    p.beta = a->beta;
    p.h0 = a->initial_state;
    p.o = a->o;
    p.ht = a->final_state;
    p.pre = pre_of(a);
    return p;
}

struct BwdLayout {
    Layout f;
    // bf16 io: records, kept states; fp32 io: the fp32 backward's own workspace and, with a gate, the
    // activated decay; with a gate, the gradient of the activated decay
    size_t keep, dg_act, act, kda_bytes, E, G, PHI, total;
    Segments seg;
};

size_t keep_bytes(int K, int V)
{
    return K == 64 ? (V == 64 ? Keep<64, 64>::BYTES : Keep<64, 128>::BYTES)
                   : (V == 64 ? Keep<128, 64>::BYTES : Keep<128, 128>::BYTES);
}

// fp32 io: the arguments of kda::run_backward (g: the activated decay).
kda_fwd_args f32_args(const gdn_args *a, const float *g)
{
    kda_fwd_args w = {};
    w.B = a->B;
    w.T = a->T;
    w.N = a->N;
    w.H = a->H;
    w.HV = a->HV;
    w.K = a->K;
    w.V = a->V;
    w.io = KDA_FP32;
    w.q = a->q;
    w.k = a->k;
    w.v = a->v;
    w.g = g;
    w.beta = a->beta;
    w.scale = a->scale;
    w.cu_seqlens = a->cu_seqlens;
    w.initial_state = a->initial_state;
    w.qk_l2norm = a->qk_l2norm;
    w.beta_sigmoid = a->beta_sigmoid;
    return w;
}

BwdLayout bwd_layout(const gdn_args *a)
{
    BwdLayout L = {};
    L.f = layout(a);
    const size_t slots = (size_t)L.f.slots * a->HV, rows = (size_t)L.f.tt * a->HV;
    size_t at;
    if (a->io == KDA_BF16) {
        L.keep = slots * RecB::BYTES;
        L.E = L.keep + slots * keep_bytes(a->K, a->V);
        L.seg = plan_segments(L.f.tt, a->N, a->cu_seqlens != nullptr, a->HV, a->K, 2 * (a->V / 64), 2,
                              ChunkTimes{6.0, 7.0, 4.0});
        const size_t ends = (size_t)L.seg.slots * a->HV * a->K * 4;
        L.G = L.E + ends * a->V;
        L.PHI = L.G + ends * a->V;
        at = L.PHI + 2 * ends * a->K;
    } else {
        const kda_fwd_args w = f32_args(a, nullptr);
        L.kda_bytes = kda_bwd_workspace_bytes(&w);
        L.act = align256(L.kda_bytes);
        at = L.act + (a->gate != KDA_GATE_NONE ? align256(rows * 4) : 0);
    }
    L.dg_act = at;
    L.total = at + (a->gate != KDA_GATE_NONE ? align256(rows * 4) : 0);
    return L;
}

// gdn_bwd's arguments but q, k, v and the workspace.
kda_status check_bwd(const gdn_args *a, const void *d_o, const float *dht, const void *dq, const void *dk,
                     const void *dv, const void *dg, const void *dbeta, const float *dh0,
                     const float *dA_log, const float *ddt_bias)
{
    kda_status st = check_chunks(a);
    if (st != KDA_OK || (st = check_pre(a)) != KDA_OK) return st;
    if (a->gate != KDA_GATE_NONE && (!dA_log || !aligned(dA_log, 4) || !aligned(ddt_bias, 4)))
        return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {a->g, a->beta, d_o, dq, dk, dv, dg, dbeta};
    if ((int64_t)a->B * a->T > 0)
        for (const void *p : ptrs)
            if (!p || !aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    const void *opt[] = {a->initial_state, a->cu_seqlens, dht, dh0};
    for (const void *p : opt)
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

}  // namespace

extern "C" {

size_t gdn_bwd_workspace_bytes(const gdn_args *a)
{
    if (check_chunks(a) != KDA_OK) return 0;
    const BwdLayout L = bwd_layout(a);
    return a->io == KDA_FP32 && L.kda_bytes == 0 ? 0 : L.total;
}

kda_status gdn_bwd(const gdn_args *a, const void *d_o, const float *dht, void *workspace,
                   size_t ws_bytes, void *dq, void *dk, void *dv, void *dg, void *dbeta,
                   float *dh0, float *dA_log, float *ddt_bias, void *stream)
{
    kda_status st = check_bwd(a, d_o, dht, dq, dk, dv, dg, dbeta, dh0, dA_log, ddt_bias);
    if (st != KDA_OK) return st;
    const bool gated = a->gate != KDA_GATE_NONE, f32 = a->io == KDA_FP32;
    const BwdLayout L = bwd_layout(a);
    const void *qkv[] = {a->q, a->k, a->v};
    if (L.f.tt > 0)
        for (const void *p : qkv)
            if (!p || !aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    if (f32 && L.kda_bytes == 0) return KDA_ERR_UNSUPPORTED;
    if (L.f.tt > 0 && (!workspace || ws_bytes < L.total || !aligned(workspace, 256)))
        return KDA_ERR_WORKSPACE;
    uint8_t *const ws = (uint8_t *)workspace;
    hipStream_t hs = (hipStream_t)stream;
    Params p = params_of(a, L.f);
    p.rec = ws;
    float *const dg_act = gated ? (float *)(ws + L.dg_act) : nullptr;
    hipError_t e;
    if (f32) {
        float *const act = gated ? (float *)(ws + L.act) : nullptr;
        if (gated && launch_activate_decay(p, act, hs) != hipSuccess) return KDA_ERR_HIP;
        const kda_fwd_args w = f32_args(a, gated ? act : (const float *)a->g);
        st = kda::run_backward(&w, true, d_o, dht, ws, L.kda_bytes, (float *)dq, (float *)dk, (float *)dv,
                               gated ? dg_act : (float *)dg, (float *)dbeta, dh0, nullptr, nullptr, stream);
        if (st != KDA_OK) return st;
        e = hipSuccess;
    } else {
        if (L.f.tt > 0) {
            e = a->K == 64 ? launch_prepare_bwd<64>(p, hs) : launch_prepare_bwd<128>(p, hs);
            if (e != hipSuccess) return KDA_ERR_HIP;
        }
        BwdParams b = {};
        b.f = p;
        b.f.seg = L.seg;
        b.f.seg.E = (float *)(ws + L.E);
        b.f.seg.G = (float *)(ws + L.G);
        b.f.seg.PHI = (float *)(ws + L.PHI);
        b.d_o = (const uint16_t *)d_o;
        b.dht = dht;
        b.keep = ws + L.keep;
        b.dq = (uint16_t *)dq;
        b.dk = (uint16_t *)dk;
        b.dv = (uint16_t *)dv;
        b.dbeta = (uint16_t *)dbeta;
        b.dg = (uint16_t *)dg;
        b.dg_act = dg_act;
        b.dh0 = dh0;
        e = by_dims(a->K, a->V, [&](auto k, auto v) {
            return launch_backward<decltype(k)::value, decltype(v)::value>(b, hs);
        });
    }
    if (e == hipSuccess && gated)
        e = launch_gate_backward(p, f32, dg_act, dg, dA_log, ddt_bias, hs);
    return e == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t gdn_bwd_packed_workspace_bytes(const gdn_args *a)
{
    const size_t need = gdn_bwd_workspace_bytes(a);
    if (need == 0) return 0;
    const size_t e = a->io == KDA_FP32 ? 4 : 2, tt = (size_t)a->B * a->T;
    return align256(need) + 2 * align256(tt * a->H * a->K * e) + align256(tt * a->HV * a->V * e);
}

kda_status gdn_bwd_packed(const gdn_args *a, const float *q_scale, const float *k_scale,
                          const float *v_scale, const void *d_o, const float *dht, void *workspace,
                          size_t ws_bytes, void *dq, void *dk, void *dv, void *dg, void *dbeta,
                          float *dh0, float *dA_log, float *ddt_bias, void *stream)
{
    const kda_status st = check_bwd(a, d_o, dht, dq, dk, dv, dg, dbeta, dh0, dA_log, ddt_bias);
    if (st != KDA_OK) return st;
    const size_t need = align256(gdn_bwd_workspace_bytes(a)), total = gdn_bwd_packed_workspace_bytes(a);
    const int64_t tt = (int64_t)a->B * a->T;
    gdn_args b = *a;
    if (tt > 0) {
        const float *const scale[3] = {q_scale, k_scale, v_scale};
        const int8_t *const data[3] = {(const int8_t *)a->q, (const int8_t *)a->k, (const int8_t *)a->v};
        for (int i = 0; i < 3; ++i)
            if (!data[i] || !scale[i] || !aligned(data[i], 16) || !aligned(scale[i], 4)) return KDA_ERR_INVALID_ARG;
        // four values a lane, less than 2^32 lanes
        if (total == 0 || tt * (2 * a->H * a->K + a->HV * a->V) >= (int64_t)1 << 33) return KDA_ERR_UNSUPPORTED;
        if (!workspace || ws_bytes < total || !aligned(workspace, 256)) return KDA_ERR_WORKSPACE;
        const size_t e = a->io == KDA_FP32 ? 4 : 2, qk = align256((size_t)tt * a->H * a->K * e);
        uint8_t *const at = (uint8_t *)workspace + need;
        void *const x[3] = {at, at + qk, at + 2 * qk};
        b.q = x[0];
        b.k = x[1];
        b.v = x[2];
        const int64_t rows[3] = {tt * a->H, tt * a->H, tt * a->HV};
        const int32_t D[3] = {a->K, a->K, a->V};
        if (launch_unpack3(data, scale, rows, D, x, a->io == KDA_FP32, (hipStream_t)stream) != hipSuccess)
            return KDA_ERR_HIP;
    }
    return gdn_bwd(&b, d_o, dht, workspace, need, dq, dk, dv, dg, dbeta, dh0, dA_log, ddt_bias, stream);
}

size_t gdn_fwd_workspace_bytes(const gdn_args *a)
{
    if (check_chunks(a) != KDA_OK || recurrent(a)) return 0;
    return layout(a).total;
}

kda_status gdn_fwd(const gdn_args *a, void *workspace, size_t ws_bytes, void *stream)
{
    kda_status st = check_shapes(a);
    if (st != KDA_OK) return st;
    if ((st = check_tensors(a)) != KDA_OK) return st;
    hipStream_t hs = (hipStream_t)stream;
    if (recurrent(a)) return run_recurrent(a, a->initial_state, a->final_state, nullptr, 0, hs);
    if ((st = check_chunks(a)) != KDA_OK) return st;
    const Layout L = layout(a);
    if (L.tt > 0 && (!workspace || ws_bytes < L.total || !aligned(workspace, 256)))
        return KDA_ERR_WORKSPACE;
    uint8_t *const ws = (uint8_t *)workspace;
    const bool f32 = a->io == KDA_FP32;
    Params p = params_of(a, L);
    p.rec = ws;
    p.seg = L.seg;
    p.seg.E = (float *)(ws + L.E);
    p.seg.PHI = (float *)(ws + L.PHI);
    if (f32 && L.tt > 0) {
        const int64_t n = L.tt * a->H * a->K;
        if (launch_split_planes((const float *)a->q, (const float *)a->k, n, (uint16_t *)(ws + L.q),
                                (uint16_t *)(ws + L.k), hs) != hipSuccess)
            return KDA_ERR_HIP;
        for (int i = 0; i < 3; ++i) {
            p.q[i] = (const uint16_t *)(ws + L.q) + i * n;
            p.k[i] = (const uint16_t *)(ws + L.k) + i * n;
        }
    }
    if (L.tt > 0) {
        const hipError_t e = a->K == 64 ? launch_prepare<64>(p, f32, hs) : launch_prepare<128>(p, f32, hs);
        if (e != hipSuccess) return KDA_ERR_HIP;
    }
    const hipError_t e = by_dims(a->K, a->V, [&](auto k, auto v) {
        return launch_state<decltype(k)::value, decltype(v)::value>(p, f32, hs);
    });
    return e == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

kda_status gdn_step(const gdn_args *a, float *state, const int32_t *state_indices, int32_t slots,
                    void *stream)
{
    kda_status st = check_shapes(a);
    if (st != KDA_OK) return st;
    if (a->cu_seqlens || slots < 0 || (!state_indices && slots < a->B)) return KDA_ERR_INVALID_ARG;
    if ((st = check_tensors(a)) != KDA_OK) return st;
    if (a->T == 0) return KDA_OK;
    if ((slots > 0 && !state) || !aligned(state, 16) || !aligned(state_indices, 4))
        return KDA_ERR_INVALID_ARG;
    return run_recurrent(a, state, state, state_indices, slots, (hipStream_t)stream);
}

}  // extern "C"
