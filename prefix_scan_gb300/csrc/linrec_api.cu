// linrec_api.cu -- the gated linear recurrence's C ABI: argument checks,
// workspace sizing, dispatch to the launchers.
#include <climits>
#include <cstdint>

#include "linrec_internal.h"
#include "scan_internal.h"

namespace {

ps_status done(cudaError_t e) {
    if (e == cudaSuccess) return PS_OK;
    ps::note_cuda_error(e);
    return PS_ERR_CUDA;
}
size_t real_bytes(int t) { return t == PS_REAL_F32 ? 4 : 2; }
bool known(int t) { return t == PS_REAL_F32 || t == PS_REAL_BF16 || t == PS_REAL_F16; }
long long total_tokens(const ps_linrec_shape *d) { return d->cu_seqlens ? d->tokens : d->num_seqs * d->tokens; }
long long tiles_of(const ps_linrec_shape *d) { return (total_tokens(d) + ps::kLinrecTile - 1) / ps::kLinrecTile; }
long long blocks_of(const ps_linrec_shape *d) { return (d->channels + ps::kLinrecWide - 1) / ps::kLinrecWide; }

bool valid(const ps_linrec_shape *d) {
    if (d == nullptr || !known(d->type)) return false;
    if (d->gate_type != PS_REAL_F32 && d->gate_type != d->type) return false;
    if (d->num_seqs < 0 || d->tokens < 0 || d->num_seqs > INT_MAX || d->tokens > INT_MAX) return false;
    if (d->channels < 1 || d->channels > INT_MAX) return false;
    if (reinterpret_cast<uintptr_t>(d->cu_seqlens) % 4 != 0) return false;
    if (total_tokens(d) > INT_MAX - 512) return false;
    // a ticket a tile, and in steps a CTA a sequence and part of the channels
    if (blocks_of(d) * (tiles_of(d) > 1 ? tiles_of(d) : 1) > INT_MAX) return false;
    return (d->channels + 127) / 128 * (d->num_seqs > 1 ? d->num_seqs : 1) <= INT_MAX;
}

bool tensor_ok(const ps_linrec_tensor *t, size_t es) {
    return t != nullptr && t->data != nullptr && reinterpret_cast<uintptr_t>(t->data) % es == 0;
}
// Whether every row starts on a multiple of `n` elements.
bool rows_on(const ps_linrec_tensor *t, size_t es, int n, bool packed) {
    return reinterpret_cast<uintptr_t>(t->data) % (n * es) == 0 && ((packed ? 0 : t->seq_stride) | t->tok_stride) % n == 0;
}
bool on(const void *p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
ps::LinrecTensor tensor(const ps_linrec_shape *d, const ps_linrec_tensor *t, size_t es) {
    const bool packed = d->cu_seqlens != nullptr;
    const bool flat = packed || d->num_seqs == 1 || t->seq_stride == t->tok_stride * d->tokens;
    int piece = (int)es;
    for (int bytes : {4, 16})
        if (rows_on(t, es, bytes / (int)es, packed) && d->channels % (bytes / (int)es) == 0) piece = bytes;
    return {t->data, packed ? 0 : (long long)t->seq_stride, (long long)t->tok_stride, flat, piece};
}

struct Range {
    uintptr_t a, b;
};
Range range(const void *p, size_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, p ? a + bytes : a};
}
// The bytes that a strided tensor spans.
Range range(const ps_linrec_shape *d, const ps_linrec_tensor *t, size_t es) {
    int64_t lo = 0, hi = 0;
    auto reach = [&](int64_t stride, int64_t n) {
        if (n > 0) (stride < 0 ? lo : hi) += stride * (n - 1);
    };
    if (d->cu_seqlens == nullptr) reach(t->seq_stride, d->num_seqs);
    reach(t->tok_stride, d->tokens);
    const uintptr_t p = reinterpret_cast<uintptr_t>(t->data);
    return {p + lo * (int64_t)es, p + (hi + d->channels) * (int64_t)es};
}
bool meet(const Range &x, const Range &y) { return x.a < y.b && y.a < x.b; }
template <int NO, int NI>
bool outputs_meet(const Range (&out)[NO], const Range (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = i + 1; j < NO; ++j)
            if (meet(out[i], out[j])) return true;
        for (int j = 0; j < NI; ++j)
            if (meet(out[i], in[j])) return true;
    }
    return false;
}

// Ticket, maps, states, a copy of the states at the start for calls in place, and in training the states before
// the backward pass's tiles.
struct Parts {
    size_t copy, start, total;
};
size_t up(size_t n) { return (n + 255) / 256 * 256; }
Parts parts_of(const ps_linrec_shape *d, int train) {
    Parts p{};
    const size_t tiles = (size_t)tiles_of(d), places = (tiles + ps::kLinrecSlack) * (size_t)blocks_of(d) * ps::kLinrecWide;
    p.copy = tiles > 1 ? up(256 + places * 12) : 0;
    p.start = p.copy + up((size_t)d->num_seqs * (size_t)d->channels * 4);
    const size_t tokens = ps::linrec_start_tokens(real_bytes(d->type), real_bytes(d->gate_type));
    p.total = p.start + (train ? up(((size_t)total_tokens(d) + tokens - 1) / tokens * (size_t)d->channels * 4) : 0);
    return p;
}
void place(ps::LinrecArgs &a, const ps_linrec_shape *d, int train, void *ws) {
    a.blocks = (int)blocks_of(d);
    a.start_tokens = ps::linrec_start_tokens(real_bytes(d->type), real_bytes(d->gate_type));
    a.ticket = static_cast<unsigned *>(ws);
    a.start = train ? reinterpret_cast<float *>(static_cast<unsigned char *>(ws) + parts_of(d, train).start) : nullptr;
}
// Tiles read the states at the start while others write those at the end: where both have one place, the first are read
// from a copy.
cudaError_t apart(const float *&start, const float *end, const ps_linrec_shape *d, int train, void *ws, cudaStream_t s) {
    if (start == nullptr || start != end) return cudaSuccess;
    float *copy = reinterpret_cast<float *>(static_cast<unsigned char *>(ws) + parts_of(d, train).copy);
    const cudaError_t e = cudaMemcpyAsync(copy, start, (size_t)d->num_seqs * d->channels * 4, cudaMemcpyDeviceToDevice, s);
    start = copy;
    return e;
}
// Without tokens every sequence is empty and hands its state on.
cudaError_t hand_on(const float *from, float *to, size_t bytes, cudaStream_t s) {
    if (to == nullptr || to == from) return cudaSuccess;
    return from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(to, 0, bytes, s);
}

}  // namespace

bool ps::linrec_tensor_map(CUtensorMap &map, const LinrecTensor &x, const LinrecArgs &a, size_t bytes, bool f16, int runs, int run) {
    typedef CUresult (*Encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                               const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    const long long row = x.tok * (long long)bytes;
    if (encode == nullptr || !x.flat || row % 16 != 0 || row <= 0 || row * run >= 1ll << 40 || !on(x.p, 16) || a.total < run)
        return false;
    const cuuint64_t sizes[3] = {(cuuint64_t)a.channels, (cuuint64_t)(a.total / run), (cuuint64_t)run};
    const cuuint64_t strides[2] = {(cuuint64_t)(row * run), (cuuint64_t)row};
    const cuuint32_t box[3] = {(cuuint32_t)kLinrecWide, (cuuint32_t)runs, (cuuint32_t)run}, steps[3] = {1, 1, 1};
    const CUtensorMapDataType type = bytes == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : f16      ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return encode(&map, type, 3, const_cast<void *>(x.p), sizes, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

extern "C" size_t ps_linrec_workspace_size(const ps_linrec_shape *d, int train) {
    if (!valid(d) || d->num_seqs == 0) return 0;
    return parts_of(d, train).total;
}

extern "C" ps_status ps_linrec_forward(const ps_linrec_shape *d, const ps_linrec_tensor *x, const ps_linrec_tensor *g,
                                       const float *h0, float *ht, void *h, int train, void *ws, size_t ws_bytes,
                                       ps_stream_t stream) {
    if (!valid(d)) return PS_ERR_INVALID_ARG;
    if (d->num_seqs == 0) return PS_OK;
    const size_t es = real_bytes(d->type), gs = real_bytes(d->gate_type), need = ps_linrec_workspace_size(d, train);
    const size_t states = (size_t)d->num_seqs * d->channels * 4;
    const long long total = total_tokens(d);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!on(h0, 4) || !on(ht, 4)) return PS_ERR_INVALID_ARG;
    if (h0 != nullptr && h0 == ht && train) return PS_ERR_OVERLAP;
    if (total == 0) {
        const Range in[] = {range(h0 == ht ? nullptr : h0, states)}, out[] = {range(ht, states)};
        if (outputs_meet(out, in)) return PS_ERR_OVERLAP;
        return done(hand_on(h0, ht, states, s));
    }
    if (!tensor_ok(x, es) || !tensor_ok(g, gs)) return PS_ERR_INVALID_ARG;
    if (h == nullptr || !on(h, es) || ws == nullptr || !on(ws, 256)) return PS_ERR_INVALID_ARG;
    if (ws_bytes < need) return PS_ERR_WORKSPACE_TOO_SMALL;
    const Range in[] = {range(d, x, es), range(d, g, gs), range(h0 == ht ? nullptr : h0, states),
                        range(d->cu_seqlens, ((size_t)d->num_seqs + 1) * 4)};
    const Range out[] = {range(h, (size_t)total * d->channels * es), range(ht, states), range(ws, need)};
    if (outputs_meet(out, in)) return PS_ERR_OVERLAP;
    ps::LinrecArgs a{};
    a.seqs = d->num_seqs;
    a.tokens = d->tokens;
    a.total = total;
    a.cu = d->cu_seqlens;
    a.channels = d->channels;
    a.x = tensor(d, x, es);
    a.g = tensor(d, g, gs);
    a.pairs = d->channels % 2 == 0 && on(h, 2 * es);
    a.h0 = h0;
    a.ht = ht;
    a.h = h;
    place(a, d, train, ws);
    cudaError_t e = apart(a.h0, ht, d, train, ws, s);
    if (e == cudaSuccess) e = ps::launch_linrec_forward(a, d->type, d->gate_type, d->tied != 0, s);
    return done(e);
}

extern "C" ps_status ps_linrec_backward(const ps_linrec_shape *d, const ps_linrec_tensor *x, const ps_linrec_tensor *g,
                                        const float *h0, const ps_linrec_tensor *d_h, const float *d_ht, void *dx, void *dg,
                                        float *dh0, void *ws, size_t ws_bytes, ps_stream_t stream) {
    if (!valid(d)) return PS_ERR_INVALID_ARG;
    if (d->num_seqs == 0) return PS_OK;
    const size_t es = real_bytes(d->type), gs = real_bytes(d->gate_type), need = ps_linrec_workspace_size(d, 1);
    const size_t states = (size_t)d->num_seqs * d->channels * 4;
    const long long total = total_tokens(d);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!on(h0, 4) || !on(d_ht, 4) || !on(dh0, 4)) return PS_ERR_INVALID_ARG;
    if (total == 0) {
        const Range in[] = {range(d_ht == dh0 ? nullptr : d_ht, states)}, out[] = {range(dh0, states)};
        if (outputs_meet(out, in)) return PS_ERR_OVERLAP;
        return done(hand_on(d_ht, dh0, states, s));
    }
    if (!tensor_ok(x, es) || !tensor_ok(g, gs) || !tensor_ok(d_h, es)) return PS_ERR_INVALID_ARG;
    if (dx == nullptr || dg == nullptr || !on(dx, es) || !on(dg, gs) || ws == nullptr || !on(ws, 256)) return PS_ERR_INVALID_ARG;
    if (ws_bytes < need) return PS_ERR_WORKSPACE_TOO_SMALL;
    const Range in[] = {range(d, x, es), range(d, g, gs), range(d, d_h, es), range(h0, states),
                        range(d_ht == dh0 ? nullptr : d_ht, states), range(d->cu_seqlens, ((size_t)d->num_seqs + 1) * 4)};
    const Range out[] = {range(dx, (size_t)total * d->channels * es), range(dg, (size_t)total * d->channels * gs),
                         range(dh0, states), range(ws, need)};
    if (outputs_meet(out, in)) return PS_ERR_OVERLAP;
    ps::LinrecArgs a{};
    a.seqs = d->num_seqs;
    a.tokens = d->tokens;
    a.total = total;
    a.cu = d->cu_seqlens;
    a.channels = d->channels;
    a.x = tensor(d, x, es);
    a.g = tensor(d, g, gs);
    a.dout = tensor(d, d_h, es);
    a.pairs = d->channels % 2 == 0 && on(dx, 2 * es) && on(dg, 2 * gs);
    a.h0 = h0;
    a.dht = d_ht;
    a.dh0 = dh0;
    a.dx = dx;
    a.dg = dg;
    place(a, d, 1, ws);
    cudaError_t e = apart(a.dht, dh0, d, 1, ws, s);
    if (e == cudaSuccess) e = ps::launch_linrec_backward(a, d->type, d->gate_type, d->tied != 0, s);
    return done(e);
}

extern "C" ps_status ps_linrec_step(const ps_linrec_shape *d, const ps_linrec_tensor *x, const ps_linrec_tensor *g,
                                    float *state, int64_t pages, const int32_t *slots, const int32_t *lengths, void *h,
                                    ps_stream_t stream) {
    if (!valid(d) || d->cu_seqlens != nullptr || pages < 0 || pages > INT_MAX) return PS_ERR_INVALID_ARG;
    if (d->num_seqs == 0 || d->tokens == 0) return PS_OK;
    const size_t es = real_bytes(d->type), gs = real_bytes(d->gate_type);
    if (!tensor_ok(x, es) || !tensor_ok(g, gs) || (state == nullptr && pages > 0) || h == nullptr || !on(h, es) || !on(state, 4) ||
        !on(slots, 4) || !on(lengths, 4))
        return PS_ERR_INVALID_ARG;
    const Range in[] = {range(d, x, es), range(d, g, gs), range(slots, (size_t)d->num_seqs * 4),
                        range(lengths, (size_t)d->num_seqs * 4)};
    const Range out[] = {range(h, (size_t)total_tokens(d) * d->channels * es), range(state, (size_t)pages * d->channels * 4)};
    if (outputs_meet(out, in)) return PS_ERR_OVERLAP;
    const bool vec = d->channels % 4 == 0 && on(h, 4 * es) && on(state, 16) && rows_on(x, es, 4, false) && rows_on(g, gs, 4, false);
    ps::LinrecStepArgs a{};
    a.seqs = d->num_seqs;
    a.pages = pages;
    a.channels = d->channels;
    a.t = (int)d->tokens;
    a.x = tensor(d, x, es);
    a.g = tensor(d, g, gs);
    a.state = state;
    a.slots = slots;
    a.lengths = lengths;
    a.h = h;
    return done(ps::launch_linrec_step(a, d->type, d->gate_type, d->tied != 0, vec, reinterpret_cast<cudaStream_t>(stream)));
}
