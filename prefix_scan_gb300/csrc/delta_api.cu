// delta_api.cu -- the gated delta rule's C ABI: argument checks, workspace
// sizing, dispatch to the launchers.
#include <climits>
#include <cstdint>

#include "delta_internal.h"
#include "scan_internal.h"

namespace {

ps_status done(cudaError_t e) {
    if (e == cudaSuccess) return PS_OK;
    ps::note_cuda_error(e);
    return PS_ERR_CUDA;
}
size_t real_bytes(int t) { return t == PS_REAL_F32 ? 4 : 2; }
bool known(int t) { return t == PS_REAL_F32 || t == PS_REAL_BF16 || t == PS_REAL_F16; }

bool valid(const ps_delta_shape *d) {
    if (d == nullptr || !known(d->type)) return false;
    if (d->beta_type != PS_REAL_F32 && d->beta_type != d->type) return false;
    if (d->num_seqs < 0 || d->tokens < 0 || d->num_seqs > INT_MAX || d->tokens > INT_MAX) return false;
    if (d->heads_k < 1 || d->heads_v < 1 || d->heads_v % d->heads_k != 0 || d->heads_v > 65535) return false;
    if (d->dim_k < 1 || d->dim_k > ps::kMaxDimK || d->dim_v < 1 || d->dim_v > 1024) return false;
    if (reinterpret_cast<uintptr_t>(d->cu_seqlens) % 4 != 0) return false;
    // grids are one-dimensional over chunks or over (sequence, head, block of columns)
    if (ps::delta_slots(d->num_seqs, d->tokens, d->cu_seqlens != nullptr) > INT_MAX / 2) return false;
    const int64_t slots = ps::delta_slots(d->num_seqs, d->tokens, d->cu_seqlens != nullptr);   // no more segments than chunks and sequences
    return (slots + d->num_seqs) <= INT_MAX / ((int64_t)d->heads_v * ((d->dim_v + 15) / 16 + 1));
}
long long total_tokens(const ps_delta_shape *d) { return d->cu_seqlens ? d->tokens : d->num_seqs * d->tokens; }

// A tensor's base is aligned to its element; no stride may take the rows of two heads or tokens
// into one another's way, but broadcast inputs (stride 0) are fine.
bool tensor_ok(const ps_delta_tensor *t, size_t es) {
    return t != nullptr && t->data != nullptr && reinterpret_cast<uintptr_t>(t->data) % es == 0;
}
bool vectors(const ps_delta_tensor &t, int dim, size_t es, bool packed) {
    const int64_t bits = (packed ? 0 : t.seq_stride) | t.tok_stride | t.head_stride;
    return dim % 8 == 0 && reinterpret_cast<uintptr_t>(t.data) % 16 == 0 && (bits * (int64_t)es) % 16 == 0;
}
ps::DeltaTensor tensor(const ps_delta_tensor *t, bool packed) {
    return {t->data, packed ? 0 : (long long)t->seq_stride, (long long)t->tok_stride, (long long)t->head_stride};
}
ps::DeltaShape shape_of(const ps_delta_shape *d) {
    return {(long long)d->num_seqs, (long long)d->tokens, d->cu_seqlens, d->heads_k, d->heads_v, d->dim_k, d->dim_v, d->scale};
}

struct Range {
    uintptr_t a, b;
};
Range range(const void *p, size_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, p ? a + bytes : a};
}
// The bytes that a strided tensor spans.
Range range(const ps_delta_shape *d, const ps_delta_tensor *t, int heads, int dim, size_t es) {
    const bool packed = d->cu_seqlens != nullptr;
    int64_t lo = 0, hi = 0;
    auto reach = [&](int64_t stride, int64_t n) {
        if (n > 0) (stride < 0 ? lo : hi) += stride * (n - 1);
    };
    if (!packed) reach(t->seq_stride, d->num_seqs);
    reach(t->tok_stride, d->tokens);
    reach(t->head_stride, heads);
    const uintptr_t p = reinterpret_cast<uintptr_t>(t->data);
    return {p + lo * (int64_t)es, p + (hi + dim) * (int64_t)es};
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

size_t state_bytes(const ps_delta_shape *d) { return (size_t)d->heads_v * d->dim_k * d->dim_v * 4; }   // of a sequence
size_t chunks_bytes(const ps_delta_shape *d, int train) {
    const long long slots = ps::delta_slots(d->num_seqs, d->tokens, d->cu_seqlens != nullptr);
    return (size_t)slots * d->heads_v * ps::chunk_layout(d->dim_k, d->dim_v, train != 0).stride;
}
// The workspace's parts after the chunks': keys and queries, what segments need, the sequences' order, and in
// training the word of a chain that gave up, 256 bytes before the end.
struct Parts {
    int seg;
    long long seg_slots;
    size_t kq, seg_m, seg_state, seg_h, order, failed, total;
    bool ordered;
};
Parts parts_of(const ps_delta_shape *d, int train) {
    const bool packed = d->cu_seqlens != nullptr;
    const long long slots = ps::delta_slots(d->num_seqs, d->tokens, packed);
    Parts p{};
    p.kq = chunks_bytes(d, train);
    p.seg_m = p.kq + (size_t)slots * d->heads_k * ps::kq_stride(d->dim_k, d->type == PS_REAL_BF16 ? 1 : 2);
    const long long chunks = packed ? d->tokens / ps::kChunk / (d->num_seqs ? d->num_seqs : 1) : (d->tokens + ps::kChunk - 1) / ps::kChunk;
    p.seg = ps::segment_chunks(d->num_seqs * d->heads_v * ps::blocks_v(d->dim_v), chunks, train != 0);
    p.seg_slots = ps::segment_slots(slots, d->num_seqs, p.seg);
    p.seg_state = p.seg_m + (size_t)p.seg_slots * d->heads_v * ps::seg_m_bytes(d->dim_k);
    p.seg_h = p.seg_state + (p.seg ? (size_t)(p.seg_slots + 1) * state_bytes(d) : 0);
    p.order = p.seg_h + (p.seg ? (size_t)d->num_seqs * state_bytes(d) : 0);
    p.ordered = packed && !p.seg && d->num_seqs > 1 && d->num_seqs <= ps::kOrdered &&
                d->num_seqs * d->heads_v * ps::blocks_v(d->dim_v) > 152;   // as many run at once
    p.failed = p.order + (p.ordered ? (size_t)d->num_seqs * 4 : 0);
    p.failed = (p.failed + 255) / 256 * 256;
    p.total = p.failed + (train && slots > 0 ? 256 : 0);
    return p;
}
void place(ps::DeltaArgs &a, const Parts &p, void *ws) {
    a.ws = static_cast<unsigned char *>(ws);
    a.kq = a.ws + p.kq;
    a.seg = p.seg;
    a.seg_slots = p.seg_slots;
    a.seg_m = a.ws + p.seg_m;
    a.seg_state = reinterpret_cast<float *>(a.ws + p.seg_state);
    a.seg_h = reinterpret_cast<float *>(a.ws + p.seg_h);
    a.order = p.ordered ? reinterpret_cast<int32_t *>(a.ws + p.order) : nullptr;
    a.failed = p.total > p.failed ? reinterpret_cast<int *>(a.ws + p.failed) : nullptr;
}
// The chain, or where sequences are cut the states of the segments, their join and the chain.  There one CTA reads the
// state at a sequence's start and another of the same launch writes the one at its end: where both have one place, the
// first is read from a copy.
template <typename Chain>
cudaError_t run_chain(ps::DeltaArgs a, int type, bool backward, Chain chain, cudaStream_t s) {
    if (a.seg) {
        cudaError_t e = cudaSuccess;
        const float *&start = backward ? a.dht : a.h0;
        if (start != nullptr && start == (backward ? a.dh0 : a.ht)) {
            e = cudaMemcpyAsync(a.seg_h, start, (size_t)(a.s.seqs * a.s.hv) * a.s.k * a.s.v * 4, cudaMemcpyDeviceToDevice, s);
            start = a.seg_h;
        }
        a.pass = ps::kPassStates;
        if (e == cudaSuccess) e = chain(a, type, s);
        if (e == cudaSuccess) e = ps::launch_delta_join(a, backward, s);
        if (e != cudaSuccess) return e;
        a.pass = ps::kPassAll;
    }
    return chain(a, type, s);
}

}  // namespace

extern "C" size_t ps_delta_workspace_size(const ps_delta_shape *d, int train) {
    if (!valid(d)) return 0;
    return parts_of(d, train).total;
}

extern "C" ps_status ps_delta_forward(const ps_delta_shape *d, const ps_delta_tensor in5[5], const float *h0, float *ht,
                                      void *o, int train, void *ws, size_t ws_bytes, ps_stream_t stream) {
    if (!valid(d) || in5 == nullptr) return PS_ERR_INVALID_ARG;
    if (d->num_seqs == 0) return PS_OK;
    const ps_delta_tensor *q = in5 + PS_DELTA_Q, *k = in5 + PS_DELTA_K, *v = in5 + PS_DELTA_V, *g = in5 + PS_DELTA_G;
    const ps_delta_tensor *beta = in5 + PS_DELTA_BETA;
    const size_t es = real_bytes(d->type), need = ps_delta_workspace_size(d, train);
    const bool packed = d->cu_seqlens != nullptr;
    const size_t state = (size_t)d->num_seqs * state_bytes(d);
    const size_t obytes = (size_t)total_tokens(d) * d->heads_v * d->dim_v * es;
    if (reinterpret_cast<uintptr_t>(h0) % 4 != 0 || reinterpret_cast<uintptr_t>(ht) % 4 != 0) return PS_ERR_INVALID_ARG;
    ps::DeltaArgs a{};
    a.s = shape_of(d);
    a.h0 = h0;
    a.ht = ht;
    if (d->tokens > 0) {
        if (!tensor_ok(q, es) || !tensor_ok(k, es) || !tensor_ok(v, es) || !tensor_ok(g, 4) ||
            !tensor_ok(beta, real_bytes(d->beta_type)))
            return PS_ERR_INVALID_ARG;
        if (o == nullptr || reinterpret_cast<uintptr_t>(o) % es != 0) return PS_ERR_INVALID_ARG;
        if (ws == nullptr || reinterpret_cast<uintptr_t>(ws) % 256 != 0) return PS_ERR_INVALID_ARG;
        if (ws_bytes < need) return PS_ERR_WORKSPACE_TOO_SMALL;
        const Range in[] = {range(d, q, d->heads_k, d->dim_k, es), range(d, k, d->heads_k, d->dim_k, es),
                            range(d, v, d->heads_v, d->dim_v, es), range(d, g, d->heads_v, 1, 4),
                            range(d, beta, d->heads_v, 1, real_bytes(d->beta_type)),
                            range(h0 == ht ? nullptr : h0, state),
                            range(d->cu_seqlens, ((size_t)d->num_seqs + 1) * 4)};
        const Range out[] = {range(o, obytes), range(ht, state), range(ws, need)};
        if (outputs_meet(out, in)) return PS_ERR_OVERLAP;
        a.q = tensor(q, packed);
        a.k = tensor(k, packed);
        a.v = tensor(v, packed);
        a.g = tensor(g, packed);
        a.beta = tensor(beta, packed);
        a.beta_f32 = d->beta_type == PS_REAL_F32;
        a.vec_qk = vectors(*q, d->dim_k, es, packed) && vectors(*k, d->dim_k, es, packed);
        a.vec_v = vectors(*v, d->dim_v, es, packed);
        a.o = o;
        place(a, parts_of(d, train), ws);
        a.slots = ps::delta_slots(d->num_seqs, d->tokens, packed);
        a.train = train != 0;
    } else {
        const Range in[] = {range(h0 == ht ? nullptr : h0, state)};
        const Range out[] = {range(ht, state)};
        if (outputs_meet(out, in)) return PS_ERR_OVERLAP;
        a.s.cu = nullptr;   // every sequence is empty: states are handed on
    }
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (a.slots > 0) {
        const cudaError_t e = ps::launch_delta_prepare(a, d->type, s);
        if (e != cudaSuccess) return done(e);
    }
    if (d->tokens == 0 && ht == nullptr) return PS_OK;
    return done(run_chain(a, d->type, false, ps::launch_delta_chain, s));
}

extern "C" ps_status ps_delta_backward(const ps_delta_shape *d, const ps_delta_tensor *q, const ps_delta_tensor *k,
                                       const ps_delta_tensor *d_o, const float *d_ht, void *dq, void *dk, void *dv,
                                       float *dg, void *dbeta, float *dh0, void *ws, size_t ws_bytes,
                                       ps_stream_t stream) {
    if (!valid(d)) return PS_ERR_INVALID_ARG;
    if (d->num_seqs == 0) return PS_OK;
    const size_t es = real_bytes(d->type), bs = real_bytes(d->beta_type), need = ps_delta_workspace_size(d, 1);
    const bool packed = d->cu_seqlens != nullptr;
    const size_t state = (size_t)d->num_seqs * state_bytes(d);
    const size_t tokens = (size_t)total_tokens(d);
    if (reinterpret_cast<uintptr_t>(d_ht) % 4 != 0 || reinterpret_cast<uintptr_t>(dh0) % 4 != 0) return PS_ERR_INVALID_ARG;
    ps::DeltaArgs a{};
    a.s = shape_of(d);
    a.dht = d_ht;
    a.dh0 = dh0;
    if (d->tokens > 0) {
        if (!tensor_ok(q, es) || !tensor_ok(k, es) || !tensor_ok(d_o, es)) return PS_ERR_INVALID_ARG;
        if (!dq || !dk || !dv || !dg || !dbeta || !ws) return PS_ERR_INVALID_ARG;
        if ((reinterpret_cast<uintptr_t>(dq) | reinterpret_cast<uintptr_t>(dk) | reinterpret_cast<uintptr_t>(dv)) % es != 0 ||
            reinterpret_cast<uintptr_t>(dg) % 4 != 0 || reinterpret_cast<uintptr_t>(dbeta) % bs != 0 ||
            reinterpret_cast<uintptr_t>(ws) % 256 != 0)
            return PS_ERR_INVALID_ARG;
        if (ws_bytes < need) return PS_ERR_WORKSPACE_TOO_SMALL;
        const Range in[] = {range(d, q, d->heads_k, d->dim_k, es), range(d, k, d->heads_k, d->dim_k, es),
                            range(d, d_o, d->heads_v, d->dim_v, es), range(d_ht == dh0 ? nullptr : d_ht, state),
                            range(d->cu_seqlens, ((size_t)d->num_seqs + 1) * 4)};
        const Range out[] = {range(dq, tokens * d->heads_k * d->dim_k * es), range(dk, tokens * d->heads_k * d->dim_k * es),
                             range(dv, tokens * d->heads_v * d->dim_v * es), range(dg, tokens * d->heads_v * 4),
                             range(dbeta, tokens * d->heads_v * bs), range(dh0, state), range(ws, need)};
        if (outputs_meet(out, in)) return PS_ERR_OVERLAP;
        a.q = tensor(q, packed);
        a.k = tensor(k, packed);
        a.dout = tensor(d_o, packed);
        a.beta_f32 = d->beta_type == PS_REAL_F32;
        a.vec_qk = vectors(*q, d->dim_k, es, packed) && vectors(*k, d->dim_k, es, packed);
        a.vec_do = vectors(*d_o, d->dim_v, es, packed);
        a.dq = dq;
        a.dk = dk;
        a.dv = dv;
        a.dg = dg;
        a.dbeta = dbeta;
        place(a, parts_of(d, 1), ws);
        a.slots = ps::delta_slots(d->num_seqs, d->tokens, packed);
        a.train = 1;
    } else {
        const Range in[] = {range(d_ht == dh0 ? nullptr : d_ht, state)};
        const Range out[] = {range(dh0, state)};
        if (outputs_meet(out, in)) return PS_ERR_OVERLAP;
        if (dh0 == nullptr) return PS_OK;
        a.s.cu = nullptr;
    }
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = run_chain(a, d->type, true, ps::launch_delta_chain_backward, s);
    if (e == cudaSuccess && a.slots > 0) e = ps::launch_delta_gradients(a, d->type, s);
    return done(e);
}

extern "C" ps_status ps_delta_step(const ps_delta_shape *d, const ps_delta_tensor in5[5], float *state, int64_t pages,
                                   const int32_t *slots, const int32_t *lengths, void *o, ps_stream_t stream) {
    if (!valid(d) || in5 == nullptr || d->cu_seqlens != nullptr || pages < 0) return PS_ERR_INVALID_ARG;
    if (d->num_seqs == 0 || d->tokens == 0) return PS_OK;
    const ps_delta_tensor *q = in5 + PS_DELTA_Q, *k = in5 + PS_DELTA_K, *v = in5 + PS_DELTA_V, *g = in5 + PS_DELTA_G;
    const ps_delta_tensor *beta = in5 + PS_DELTA_BETA;
    const size_t es = real_bytes(d->type);
    if (!tensor_ok(q, es) || !tensor_ok(k, es) || !tensor_ok(v, es) || !tensor_ok(g, 4) ||
        !tensor_ok(beta, real_bytes(d->beta_type)))
        return PS_ERR_INVALID_ARG;
    if ((state == nullptr && pages > 0) || o == nullptr || reinterpret_cast<uintptr_t>(o) % es != 0) return PS_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(state) | reinterpret_cast<uintptr_t>(slots) | reinterpret_cast<uintptr_t>(lengths)) % 4 != 0)
        return PS_ERR_INVALID_ARG;
    const Range in[] = {range(d, q, d->heads_k, d->dim_k, es), range(d, k, d->heads_k, d->dim_k, es),
                        range(d, v, d->heads_v, d->dim_v, es), range(d, g, d->heads_v, 1, 4),
                        range(d, beta, d->heads_v, 1, real_bytes(d->beta_type)),
                        range(slots, (size_t)d->num_seqs * 4), range(lengths, (size_t)d->num_seqs * 4)};
    const Range out[] = {range(o, (size_t)total_tokens(d) * d->heads_v * d->dim_v * es),
                         range(state, (size_t)pages * d->heads_v * d->dim_k * d->dim_v * 4)};
    if (outputs_meet(out, in)) return PS_ERR_OVERLAP;
    ps::DeltaStepArgs a{};
    a.seqs = d->num_seqs;
    a.pages = pages;
    a.t = (int)d->tokens;
    a.hk = d->heads_k;
    a.hv = d->heads_v;
    a.k = d->dim_k;
    a.v = d->dim_v;
    a.scale = d->scale;
    a.q = tensor(q, false);
    a.kk = tensor(k, false);
    a.vv = tensor(v, false);
    a.g = tensor(g, false);
    a.beta = tensor(beta, false);
    a.beta_f32 = d->beta_type == PS_REAL_F32;
    a.state = state;
    a.slots = slots;
    a.lengths = lengths;
    a.o = o;
    return done(ps::launch_delta_step(a, d->type, reinterpret_cast<cudaStream_t>(stream)));
}
