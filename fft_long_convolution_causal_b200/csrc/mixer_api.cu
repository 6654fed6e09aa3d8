// mixer_api.cu -- the extern "C" boundary of the sequence-mixer operators:
// argument checks, plans and their tables, dispatch to the kernels.
#include <math.h>
#include <string.h>

#include <new>
#include <vector>

#include "mixer.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool valid_dtype(int d) { return d == FFTCONV_F32 || d == FFTCONV_BF16; }
int esize(int dtype) { return dtype == FFTCONV_BF16 ? 2 : 4; }

bool on_device(int device) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return dev == device;
}

void current_device(int* device, int* sms) {
    if (cudaGetDevice(device) != cudaSuccess ||
        cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *device) != cudaSuccess) {
        cudaGetLastError();
        *sms = 1;
    }
}

fftconv_status status_of(cudaError_t e) {
    return e == cudaSuccess ? FFTCONV_OK : e == cudaErrorNotSupported ? FFTCONV_ERR_UNSUPPORTED : FFTCONV_ERR_CUDA;
}

// device copy of a host block
fftconv_status upload(const void* host, size_t bytes, void** out) {
    void* d = nullptr;
    if (cudaMalloc(&d, bytes) != cudaSuccess) {
        cudaGetLastError();
        return FFTCONV_ERR_OOM;
    }
    if (cudaMemcpy(d, host, bytes, cudaMemcpyHostToDevice) != cudaSuccess) {
        cudaGetLastError();
        cudaFree(d);
        return FFTCONV_ERR_CUDA;
    }
    *out = d;
    return FFTCONV_OK;
}

bool multiple(const fftconv_strides& s, int64_t m) { return s.batch % m == 0 && s.head % m == 0 && s.token % m == 0; }
bool distinct(const fftconv_strides& s, int64_t B, int64_t H, int64_t N) {
    return (B == 1 || s.batch != 0) && (H == 1 || s.head != 0) && (N == 1 || s.token != 0);
}
// a tensor a pass reads or writes: 16-byte pieces everywhere
bool tokens_ok(const void* p, const fftconv_strides& s, int es) { return p && aligned16(p) && multiple(s, 16 / es); }

}  // namespace

extern "C" {

fftconv_status fftconv_linattn_plan_create(fftconv_linattn** out, int B, int H, int64_t N, int dk, int dv,
                                           fftconv_dtype dtype, const double* log_decay) {
    if (!out) return FFTCONV_ERR_INVALID_ARG;
    *out = nullptr;
    if (B < 1 || H < 1 || N < 1 || !valid_dtype(dtype) || !log_decay) return FFTCONV_ERR_INVALID_ARG;
    for (int h = 0; h < H; ++h)
        if (!(log_decay[h] <= 0.0)) return FFTCONV_ERR_INVALID_ARG;  // NaN too
    if (dk < 8 || dv < 8 || dk > FFTCONV_LINATTN_MAX_DIM || dv > FFTCONV_LINATTN_MAX_DIM || dk % 8 || dv % 8 ||
        (int64_t)B * H > 65535)
        return FFTCONV_ERR_UNSUPPORTED;
    fftconv_linattn_s* p = new (std::nothrow) fftconv_linattn_s();
    if (!p) return FFTCONV_ERR_OOM;
    p->B = B, p->H = H, p->N = N, p->dk = dk, p->dv = dv, p->dtype = dtype;
    current_device(&p->device, &p->sms);
    // [H] logarithms, [H][kLaPowers] powers (computed in fp64) rounded and in two parts, the status word
    const size_t n = (size_t)H * fftc::kLaPowers, off_pow = (size_t)H * sizeof(double),
                 off_decay = (off_pow + n * sizeof(float) + 7) / 8 * 8, off_err = off_decay + n * sizeof(float2);
    try {
        std::vector<unsigned char> host(off_err + 16, 0);
        memcpy(&host[0], log_decay, off_pow);
        for (size_t i = 0; i < n; ++i) {
            const size_t h = i / fftc::kLaPowers, e = i % fftc::kLaPowers;
            const double a = e == 0 ? 1.0 : exp(log_decay[h] * (double)e);
            const float near = (float)a;
            // The first part is rounded down, so that the second is positive, and the second never zero where that
            // changes nothing: an infinite state then stays one (no infinity of the other sign, no 0 x infinity).
            const float hi = near > a ? nextafterf(near, 0.f) : near;
            float lo = (float)(a - hi);
            if (hi >= 0x1p-100f) lo = fmaxf(lo, 0x1p-149f);
            const float2 parts = make_float2(hi, lo);
            memcpy(&host[off_pow + i * sizeof(float)], &near, sizeof(float));
            memcpy(&host[off_decay + i * sizeof(float2)], &parts, sizeof(float2));
        }
        const fftconv_status st = upload(host.data(), host.size(), &p->block);
        if (st != FFTCONV_OK) {
            delete p;
            return st;
        }
    } catch (...) {
        delete p;
        return FFTCONV_ERR_OOM;
    }
    p->d_log = (const double*)p->block;
    p->d_pow = (const float*)((const unsigned char*)p->block + off_pow);
    p->d_decay = (const float2*)((const unsigned char*)p->block + off_decay);
    p->d_err = (int*)((unsigned char*)p->block + off_err);
    *out = p;
    return FFTCONV_OK;
}

fftconv_status fftconv_linattn_plan_destroy(fftconv_linattn* p) {
    if (!p) return FFTCONV_OK;
    const cudaError_t e = p->block ? cudaFree(p->block) : cudaSuccess;
    if (e != cudaSuccess) cudaGetLastError();
    delete p;
    return status_of(e);
}

size_t fftconv_linattn_workspace_bytes(const fftconv_linattn* p, int backward) {
    return p ? fftc::la_workspace_floats(*p, backward ? 3 : 1) * sizeof(float) : 0;
}

fftconv_status fftconv_linattn_fwd(const fftconv_linattn* p, const fftconv_linattn_args* a, void* workspace,
                                   void* stream) {
    if (!p || !a || a->size != sizeof(*a) || a->B < 1 || a->B > p->B || a->N < 1 || a->N > p->N ||
        !isfinite((float)a->scale) || !on_device(p->device))
        return FFTCONV_ERR_INVALID_ARG;
    const int es = esize(p->dtype);
    if (!tokens_ok(a->q, a->sq, es) || !tokens_ok(a->k, a->sk, es) || !tokens_ok(a->v, a->sv, es) ||
        !tokens_ok(a->o, a->so, es) || !distinct(a->so, a->B, p->H, a->N) || a->o == a->q || a->o == a->k || a->o == a->v)
        return FFTCONV_ERR_INVALID_ARG;
    if (!aligned4(a->lengths) || !aligned16(a->state_in) || !aligned16(a->state_out) || !aligned16(workspace) ||
        (!workspace && fftconv_linattn_workspace_bytes(p, 0)))
        return FFTCONV_ERR_INVALID_ARG;
    const float scale = (float)a->scale;
    fftc::LaCall c;
    c.passes = 1;
    c.B = a->B, c.H = p->H, c.N = a->N, c.lengths = a->lengths, c.work = (float*)workspace;
    c.pass[0] = {a->q, a->k, a->v, a->o, a->sq, a->sk, a->sv, a->so, p->dk, p->dv, 0,
                 a->state_in, a->state_out, 0, scale, scale, 1.f};
    return status_of(fftc::launch_la(*p, c, (cudaStream_t)stream));
}

fftconv_status fftconv_linattn_bwd(const fftconv_linattn* p, const fftconv_linattn_bwd_args* a, void* workspace,
                                   void* stream) {
    if (!p || !a || a->size != sizeof(*a) || a->B < 1 || a->B > p->B || a->N < 1 || a->N > p->N ||
        !isfinite((float)a->scale) || !on_device(p->device))
        return FFTCONV_ERR_INVALID_ARG;
    const int es = esize(p->dtype);
    if (!tokens_ok(a->d_o, a->sdo, es) || !tokens_ok(a->q, a->sq, es) || !tokens_ok(a->k, a->sk, es) ||
        !tokens_ok(a->v, a->sv, es) || !tokens_ok(a->dq, a->sdq, es) || !tokens_ok(a->dk, a->sdk, es) ||
        !tokens_ok(a->dv, a->sdv, es) || !distinct(a->sdq, a->B, p->H, a->N) || !distinct(a->sdk, a->B, p->H, a->N) ||
        !distinct(a->sdv, a->B, p->H, a->N))
        return FFTCONV_ERR_INVALID_ARG;
    const void* in[4] = {a->d_o, a->q, a->k, a->v};
    for (const void* x : in)
        if (a->dq == x || a->dk == x || a->dv == x) return FFTCONV_ERR_INVALID_ARG;
    if (a->dq == a->dk || a->dk == a->dv || a->dq == a->dv) return FFTCONV_ERR_INVALID_ARG;
    if (!aligned4(a->lengths) || !aligned16(a->state_in) || !aligned16(a->d_state) || !aligned16(a->d_state_in) ||
        !aligned16(workspace) || (!workspace && fftconv_linattn_workspace_bytes(p, 1)) ||
        (a->d_state_in && (a->d_state_in == a->d_state || a->d_state_in == a->state_in)))
        return FFTCONV_ERR_INVALID_ARG;
    const float scale = (float)a->scale;
    fftc::LaCall c;
    c.passes = 3;
    c.B = a->B, c.H = p->H, c.N = a->N, c.lengths = a->lengths, c.work = (float*)workspace;
    c.pass[0] = {a->d_o, a->v, a->k, a->dq, a->sdo, a->sv, a->sk, a->sdq, p->dv, p->dk, 0,
                 a->state_in, nullptr, 1, scale, scale, 1.f};
    c.pass[1] = {a->v, a->d_o, a->q, a->dk, a->sv, a->sdo, a->sq, a->sdk, p->dv, p->dk, 1,
                 a->d_state, nullptr, 1, scale, 1.f, scale};
    c.pass[2] = {a->k, a->q, a->d_o, a->dv, a->sk, a->sq, a->sdo, a->sdv, p->dk, p->dv, 1,
                 a->d_state, a->d_state_in, 0, scale, 1.f, scale};
    return status_of(fftc::launch_la(*p, c, (cudaStream_t)stream));
}

fftconv_status fftconv_linattn_step(const fftconv_linattn* p, const fftconv_linattn_step_args* a, void* stream) {
    if (!p || !a || a->size != sizeof(*a) || a->B < 1 || a->B > p->B || a->slots_n < 1 || !isfinite((float)a->scale) ||
        !a->q || !a->k || !a->v || !a->o || !a->state || !aligned16(a->state) || !aligned4(a->slots) ||
        (!a->slots && a->slots_n < a->B) || !distinct(a->so, a->B, p->H, 1) || !on_device(p->device))
        return FFTCONV_ERR_INVALID_ARG;
    const uintptr_t mis = ((uintptr_t)a->q | (uintptr_t)a->k | (uintptr_t)a->v | (uintptr_t)a->o) & (esize(p->dtype) - 1);
    if (mis) return FFTCONV_ERR_INVALID_ARG;
    const fftc::LaStep c{a->q, a->k, a->v, a->o, a->sq.batch, a->sq.head, a->sk.batch, a->sk.head,
                         a->sv.batch, a->sv.head, a->so.batch, a->so.head, a->state, a->slots, a->B, a->slots_n,
                         (float)a->scale};
    return status_of(fftc::launch_la_step(*p, c, (cudaStream_t)stream));
}

fftconv_status fftconv_linattn_set_wait_limit(fftconv_linattn* p, uint32_t probes) {
    if (!p) return FFTCONV_ERR_INVALID_ARG;
    p->wait_limit = probes;
    return FFTCONV_OK;
}

fftconv_status fftconv_linattn_device_status(fftconv_linattn* p, void* stream) {
    if (!p || !on_device(p->device)) return FFTCONV_ERR_INVALID_ARG;
    int word = 0;
    const int zero = 0;
    if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess ||
        cudaMemcpy(&word, p->d_err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess)
        return FFTCONV_ERR_CUDA;
    if (!word) return FFTCONV_OK;
    if (cudaMemcpy(p->d_err, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess) return FFTCONV_ERR_CUDA;
    return FFTCONV_ERR_TIMEOUT;
}

fftconv_status fftconv_rotary_plan_create(fftconv_rotary** out, fftconv_dtype dtype, const fftconv_rotary_options* o) {
    if (!out) return FFTCONV_ERR_INVALID_ARG;
    *out = nullptr;
    if (!o || o->size != sizeof(*o) || !valid_dtype(dtype) || o->rot < 2 || o->rot % 2 || o->dim < o->rot ||
        o->scaling < FFTCONV_ROTARY_NONE || o->scaling > FFTCONV_ROTARY_PARTS || !(o->base > 1.0) ||
        !isfinite(o->base) || !(o->factor >= 1.0) || !isfinite(o->factor) ||
        (o->scaling == FFTCONV_ROTARY_PARTS && (!(o->context > 0.0) || !isfinite(o->context))) ||
        (o->scaling == FFTCONV_ROTARY_BASE && o->rot < 4))
        return FFTCONV_ERR_INVALID_ARG;
    if (o->dim > FFTCONV_ROTARY_MAX_DIM) return FFTCONV_ERR_UNSUPPORTED;
    const int half = o->rot / 2;
    const double base =
        o->scaling == FFTCONV_ROTARY_BASE ? o->base * pow(o->factor, o->rot / (o->rot - 2.0)) : o->base;
    // pair index (real) that turns n times over the context
    auto index_of = [&](double n) { return o->rot * log(o->context / (2.0 * M_PI * n)) / (2.0 * log(o->base)); };
    double lo = 0.0, hi = 0.0;
    if (o->scaling == FFTCONV_ROTARY_PARTS) {
        lo = fmax(0.0, floor(index_of(32.0)));
        hi = fmin(o->rot - 1.0, ceil(index_of(1.0)));
    }
    fftconv_rotary_s* p = new (std::nothrow) fftconv_rotary_s();
    if (!p) return FFTCONV_ERR_OOM;
    p->dim = o->dim, p->rot = o->rot, p->interleaved = o->interleaved ? 1 : 0, p->dtype = dtype;
    p->magnitude = o->scaling == FFTCONV_ROTARY_PARTS ? (float)(0.1 * log(o->factor) + 1.0) : 1.f;
    current_device(&p->device, &p->sms);
    uint64_t turns[FFTCONV_ROTARY_MAX_DIM / 2];
    for (int i = 0; i < half; ++i) {
        // in extended precision: the table's error times a far position is the angle's error
        long double f = powl((long double)base, -2.0L * i / o->rot);
        if (o->scaling == FFTCONV_ROTARY_LINEAR) f /= o->factor;
        if (o->scaling == FFTCONV_ROTARY_PARTS) {
            const long double keep = 1.0L - fmin(1.0, fmax(0.0, (i - lo) / fmax(hi - lo, 1e-3)));
            f = f / o->factor * (1.0L - keep) + f * keep;
        }
        f /= 2.0L * 3.14159265358979323846264338327950288L;  // turns per position, < 1 / 6
        turns[i] = (uint64_t)roundl(f * 18446744073709551616.0L);
    }
    const fftconv_status st = upload(turns, half * sizeof(uint64_t), (void**)&p->d_turns);
    if (st != FFTCONV_OK) {
        delete p;
        return st;
    }
    *out = p;
    return FFTCONV_OK;
}

fftconv_status fftconv_rotary_plan_destroy(fftconv_rotary* p) {
    if (!p) return FFTCONV_OK;
    const cudaError_t e = cudaFree(p->d_turns);
    if (e != cudaSuccess) cudaGetLastError();
    delete p;
    return status_of(e);
}

fftconv_status fftconv_rotary_apply(const fftconv_rotary* p, const fftconv_rotary_args* a, void* stream) {
    if (!p || !a || a->size != sizeof(*a) || a->B < 1 || a->N < 1 || a->H < 1 || a->H2 < 0 || !a->positions ||
        (reinterpret_cast<uintptr_t>(a->positions) & 7u) || a->position_stride < 0 || !a->x || !a->y ||
        (a->H2 && (!a->x2 || !a->y2)) || !on_device(p->device))
        return FFTCONV_ERR_INVALID_ARG;
    const uintptr_t mis = ((uintptr_t)a->x | (uintptr_t)a->y | (uintptr_t)(a->H2 ? a->x2 : nullptr) |
                           (uintptr_t)(a->H2 ? a->y2 : nullptr)) & (esize(p->dtype) - 1);
    if (mis || !distinct(a->sy, a->B, a->H, a->N) || (a->H2 && !distinct(a->sy2, a->B, a->H2, a->N)))
        return FFTCONV_ERR_INVALID_ARG;
    auto same = [](const fftconv_strides& s, const fftconv_strides& t) {
        return s.batch == t.batch && s.head == t.head && s.token == t.token;
    };
    if ((a->x == a->y && !same(a->sx, a->sy)) || (a->H2 && a->x2 == a->y2 && !same(a->sx2, a->sy2)))
        return FFTCONV_ERR_INVALID_ARG;
    if (a->H2 && (a->y == a->y2 || a->y == a->x2 || a->y2 == a->x)) return FFTCONV_ERR_INVALID_ARG;  // turned twice
    if ((double)a->B * (double)a->N * p->dim > 2147483647.0 * 256.0 || (int64_t)a->H + a->H2 > 65535)
        return FFTCONV_ERR_UNSUPPORTED;  // one grid
    const fftc::RotaryView v[2] = {
        {a->x, a->y, a->H, a->sx.batch, a->sx.head, a->sx.token, a->sy.batch, a->sy.head, a->sy.token},
        {a->x2, a->y2, a->H2, a->sx2.batch, a->sx2.head, a->sx2.token, a->sy2.batch, a->sy2.head, a->sy2.token}};
    return status_of(fftc::launch_rotary(*p, v, a->H2 ? 2 : 1, a->B, a->N, a->positions, a->position_stride,
                                         a->inverse ? 1 : 0, (cudaStream_t)stream));
}

fftconv_status fftconv_norm_plan_create(fftconv_norm** out, int64_t rows, int C, int groups, fftconv_dtype dtype,
                                        const double* eps) {
    if (!out) return FFTCONV_ERR_INVALID_ARG;
    *out = nullptr;
    // in fp32 an eps that is not zero stays so (a row of one value would give 0 x infinity), and finite
    if (rows < 1 || C < 1 || groups < 1 || rows % groups || !valid_dtype(dtype) || !eps || !(*eps >= 0.0) ||
        !isfinite((float)*eps) || (*eps > 0.0 && (float)*eps == 0.f))
        return FFTCONV_ERR_INVALID_ARG;
    if (C > FFTCONV_NORM_MAX_C || groups > 65535 || rows > 2147483647) return FFTCONV_ERR_UNSUPPORTED;
    fftconv_norm_s* p = new (std::nothrow) fftconv_norm_s();
    if (!p) return FFTCONV_ERR_OOM;
    p->rows = rows, p->C = C, p->groups = groups, p->dtype = dtype, p->eps = (float)*eps;
    current_device(&p->device, &p->sms);
    *out = p;
    return FFTCONV_OK;
}

fftconv_status fftconv_norm_plan_destroy(fftconv_norm* p) {
    delete p;
    return FFTCONV_OK;
}

fftconv_status fftconv_norm_fwd(const fftconv_norm* p, int64_t rows, const void* x, const float* w, const float* b,
                                void* y, float* mean, float* rstd, void* stream) {
    if (!p || rows < 1 || rows > p->rows || rows % p->groups || !x || !w || !b || !y || !aligned16(x) ||
        !aligned16(w) || !aligned16(b) || !aligned16(y) || !aligned4(mean) || !aligned4(rstd) || !on_device(p->device))
        return FFTCONV_ERR_INVALID_ARG;
    return status_of(fftc::launch_norm_fwd(*p, rows, x, w, b, y, mean, rstd, (cudaStream_t)stream));
}

size_t fftconv_norm_bwd_workspace_bytes(const fftconv_norm* p) { return p ? fftc::norm_workspace_bytes(*p) : 0; }

fftconv_status fftconv_norm_bwd(const fftconv_norm* p, int64_t rows, const void* dy, const void* x, const float* w,
                                const float* mean, const float* rstd, void* dx, float* dw, float* db, void* workspace,
                                void* stream) {
    if (!p || rows < 1 || rows > p->rows || rows % p->groups || !dy || !x || !w || !mean || !rstd || !dx || !dw || !db ||
        !workspace || !aligned16(dy) || !aligned16(x) || !aligned16(w) || !aligned16(dx) || !aligned4(mean) ||
        !aligned4(rstd) || !aligned4(dw) || !aligned4(db) || !aligned16(workspace) || !on_device(p->device))
        return FFTCONV_ERR_INVALID_ARG;
    return status_of(fftc::launch_norm_bwd(*p, rows, dy, x, w, mean, rstd, dx, dw, db, (float*)workspace,
                                           (cudaStream_t)stream));
}

}  // extern "C"
