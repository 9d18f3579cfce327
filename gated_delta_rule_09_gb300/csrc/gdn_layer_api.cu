// C-ABI entry points of the operators around the recurrence: argument checks
// and dispatch.  See include/gdn.h for the contract of each.
#include "gdn.h"
#include "gdn_layer.h"

namespace {

// A matrix argument: `rows` rows of `bytes`, `ld` bytes apart.
struct View {
    const char *name;
    const void *p;
    int64_t rows;
    size_t bytes, ld;
};

View flat(const char *name, const void *p, size_t bytes) { return {name, p, 1, bytes, bytes}; }

bool clash(const View &a, const View &b)
{
    if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || !a.bytes || !b.bytes) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    const size_t na = (size_t)(a.rows - 1) * a.ld + a.bytes, nb = (size_t)(b.rows - 1) * b.ld + b.bytes;
    if (pa >= pb + nb || pb >= pa + na) return false;
    // Slices of the same rows: apart when their columns are.
    if (a.ld == b.ld) {
        const size_t d = (size_t)((pb >= pa ? pb - pa : a.ld - (pa - pb) % a.ld) % a.ld);
        return !(d >= a.bytes && d + b.bytes <= a.ld);
    }
    return true;
}

// Outputs against everything else; the first `nout` views are the outputs.
gdn_status_t check_overlap(const View *v, int n, int nout)
{
    for (int i = 0; i < nout; ++i)
        for (int j = i + 1; j < n; ++j)
            if (clash(v[i], v[j]))
                return gdn_fail(GDN_ERR_INVALID_ARG, "%s overlaps %s", v[i].name, v[j].name);
    return GDN_OK;
}

gdn_status_t check_alignment(const View *v, int n, size_t al)
{
    for (int i = 0; i < n; ++i)
        if (reinterpret_cast<uintptr_t>(v[i].p) % al)
            return gdn_fail(GDN_ERR_INVALID_ARG, "%s must be aligned to %zu bytes", v[i].name, al);
    return GDN_OK;
}

// Row stride and element alignment of the matrix arguments that are there.
gdn_status_t check_rows(const View *v, int n, size_t esz)
{
    for (int i = 0; i < n; ++i)
        if (v[i].p && (int64_t)v[i].ld < (int64_t)v[i].bytes)
            return gdn_fail(GDN_ERR_INVALID_ARG, "row stride of %s is less than its row (%lld < %lld elements)",
                            v[i].name, (long long)v[i].ld / (long long)esz, (long long)(v[i].bytes / esz));
    return check_alignment(v, n, esz);
}

// Kernels count tokens and sequences in 32 bits, up to a few tiles past the last.
constexpr int kMaxCount = 0x7fff0000;

gdn_status_t check_counts(int N, int T)
{
    if (N < 0 || T < 0)
        return gdn_fail(GDN_ERR_INVALID_ARG, "negative size: %d sequences, %d tokens", N, T);
    if (N > kMaxCount || T > kMaxCount)
        return gdn_fail(GDN_ERR_UNSUPPORTED, "%d sequences, %d tokens (supported: up to %d)", N, T, kMaxCount);
    return GDN_OK;
}

gdn_status_t check_types(int dtype, int act)
{
    if (dtype != GDN_F32 && dtype != GDN_BF16)
        return gdn_fail(GDN_ERR_UNSUPPORTED, "dtype %d (expected GDN_F32 or GDN_BF16)", dtype);
    if (act != GDN_ACT_NONE && act != GDN_ACT_SILU)
        return gdn_fail(GDN_ERR_UNSUPPORTED, "activation %d (expected GDN_ACT_NONE or GDN_ACT_SILU)", act);
    return GDN_OK;
}

// Pool and slots: every sequence without slots needs an entry of its own.
gdn_status_t check_pool(const void *in, const void *out, const int32_t *slots, int N, int pool)
{
    if ((in || out) && pool < 0) return gdn_fail(GDN_ERR_INVALID_ARG, "negative pool %d", pool);
    if ((in || out) && !slots && pool < N)
        return gdn_fail(GDN_ERR_INVALID_ARG, "a pool of %d states for %d sequences (pass slots)", pool, N);
    return GDN_OK;
}

gdn_status_t launched(cudaError_t e, const char *what, int launches, int path)
{
    if (e != cudaSuccess)
        return gdn_fail(GDN_ERR_CUDA, "kernel launch (%s): %s", what, cudaGetErrorString(e));
    gdn_record_launch(launches, path);
    return GDN_OK;
}

#define GDN_TRY(call)                             \
    do {                                          \
        const gdn_status_t st_ = (call);          \
        if (st_ != GDN_OK) return st_;            \
    } while (0)

gdn_status_t conv(bool step, GdnConvArgs &a, int act, int dtype, void *stream)
{
    gdn_begin_call();
    GDN_TRY(check_counts(a.N, a.T));
    if (a.channels < 1)
        return gdn_fail(GDN_ERR_INVALID_ARG, "channels must be >= 1: %d", a.channels);
    if (a.width < 1 || a.width > 8)
        return gdn_fail(GDN_ERR_UNSUPPORTED, "width %d (supported: 1 to 8)", a.width);
    GDN_TRY(check_types(dtype, act));
    if (a.cu_seqlens && a.N < 1)
        return gdn_fail(GDN_ERR_INVALID_ARG, "cu_seqlens given with %d sequences", a.N);
    const size_t esz = dtype == GDN_BF16 ? 2 : 4;
    const int64_t rows = step ? a.N : a.cu_seqlens ? a.T : (int64_t)a.N * a.T;
    const size_t row = (size_t)a.channels * esz, state = (size_t)a.pool * (a.width - 1) * row;
    if (rows > 0 && (!a.x || !a.y || !a.weight))
        return gdn_fail(GDN_ERR_INVALID_ARG, "x, weight and y must be non-NULL");
    if (step && a.N > 0 && a.width > 1 && !a.state_out)
        return gdn_fail(GDN_ERR_INVALID_ARG, "state_out must be non-NULL");
    GDN_TRY(check_pool(a.state_in, a.state_out, a.slots, a.N, a.pool));
    const View v[] = {{"y", a.y, rows, row, (size_t)a.ld_y * esz},
                      flat("state_out", a.state_out, state),
                      {"x", a.x, rows, row, (size_t)a.ld_x * esz},
                      flat("state_in", a.state_in == a.state_out ? nullptr : a.state_in, state),
                      flat("weight", a.weight, (size_t)a.channels * a.width * 4),
                      flat("bias", a.bias, (size_t)a.channels * 4),
                      flat("slots", a.slots, (size_t)a.N * 4),
                      flat("cu_seqlens", a.cu_seqlens, ((size_t)a.N + 1) * 4)};
    if (rows > 0) {
        GDN_TRY(check_rows(v, 1, esz));
        GDN_TRY(check_rows(v + 2, 1, esz));
    }
    GDN_TRY(check_alignment(v + 1, 1, esz));
    GDN_TRY(check_alignment(v + 3, 1, esz));
    GDN_TRY(check_alignment(v + 4, 4, 4));
    GDN_TRY(check_overlap(v, 8, 2));
    gdn_record_launch(0, -1);
    if (a.N == 0 || (rows == 0 && !a.state_out)) return GDN_OK;
    if (!a.state_in && !a.state_out) a.slots = nullptr;  // no pool that a slot could be past the end of
    a.act = act;
    a.dtype = dtype == GDN_BF16 ? 1 : 0;
    GDN_TRY(gdn_device_status_word(&a.status));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launched(step ? gdn_launch_conv_step(a, s) : gdn_launch_conv_fwd(a, s), "convolution", 1, 6);
}

// The arguments of a scan or step call: outputs, fp32 arrays, rows.
constexpr int kSsmViews = 13;

void ssm_views(const GdnSsmArgs &a, int64_t rows, View *v)
{
    const size_t esz = a.dtype == 1 ? 2 : 4;
    const size_t row = (size_t)a.channels * esz, bc = (size_t)a.groups * a.d_state * esz;
    const size_t per = (size_t)a.channels * a.d_state * 4, state = (size_t)a.pool * per;
    const View all[kSsmViews] = {{"y", a.y, rows, row, (size_t)a.ld_y * esz},
                                 flat("state_out", a.state_out, state),
                                 flat("state_in", a.state_in, state),
                                 flat("A", a.A, per),
                                 flat("D", a.D, (size_t)a.channels * 4),
                                 flat("delta_bias", a.delta_bias, (size_t)a.channels * 4),
                                 flat("slots", a.slots, (size_t)a.N * 4),
                                 flat("cu_seqlens", a.cu_seqlens, ((size_t)a.N + 1) * 4),
                                 {"x", a.x, rows, row, (size_t)a.ld_x * esz},
                                 {"delta", a.delta, rows, row, (size_t)a.ld_delta * esz},
                                 {"B", a.Bm, rows, bc, (size_t)a.ld_b * esz},
                                 {"C", a.Cm, rows, bc, (size_t)a.ld_c * esz},
                                 {"z", a.z, rows, row, (size_t)a.ld_z * esz}};
    for (int i = 0; i < kSsmViews; ++i) v[i] = all[i];
}

// Everything of a scan or step call but the workspace; *nothing when there is
// nothing to compute or write.
gdn_status_t check_ssm(bool step, GdnSsmArgs &a, int dtype, bool *nothing)
{
    gdn_begin_call();
    *nothing = true;
    GDN_TRY(check_counts(a.N, a.T));
    if (a.channels < 1 || a.d_state < 1 || a.groups < 1)
        return gdn_fail(GDN_ERR_INVALID_ARG, "channels, d_state and groups must be >= 1: %d, %d, %d",
                        a.channels, a.d_state, a.groups);
    if (a.channels % a.groups)
        return gdn_fail(GDN_ERR_INVALID_ARG, "%d channels are not a multiple of %d groups", a.channels,
                        a.groups);
    if (a.d_state > 128)
        return gdn_fail(GDN_ERR_UNSUPPORTED, "d_state %d (supported: 1 to 128)", a.d_state);
    if ((int64_t)a.groups * a.d_state > 0x7fffffff)
        return gdn_fail(GDN_ERR_UNSUPPORTED, "rows of B and C of %d groups x %d states (supported: up to 2^31 - 1)",
                        a.groups, a.d_state);
    GDN_TRY(check_types(dtype, GDN_ACT_NONE));
    if (a.cu_seqlens && a.N < 1)
        return gdn_fail(GDN_ERR_INVALID_ARG, "cu_seqlens given with %d sequences", a.N);
    a.dtype = dtype == GDN_BF16 ? 1 : 0;
    const size_t esz = dtype == GDN_BF16 ? 2 : 4;
    const int64_t rows = step ? a.N : a.cu_seqlens ? a.T : (int64_t)a.N * a.T;
    if (rows > 0 && (!a.x || !a.delta || !a.A || !a.Bm || !a.Cm || !a.y))
        return gdn_fail(GDN_ERR_INVALID_ARG, "x, delta, A, B, C and y must be non-NULL");
    if (step && a.N > 0 && !a.state_out)
        return gdn_fail(GDN_ERR_INVALID_ARG, "state_out must be non-NULL");
    GDN_TRY(check_pool(a.state_in, a.state_out, a.slots, a.N, a.pool));
    View v[kSsmViews];
    ssm_views(a, rows, v);
    if (a.state_in == a.state_out) v[2].p = nullptr;  // in place: state_out stands for both
    if (rows > 0) {
        GDN_TRY(check_rows(v, 1, esz));
        GDN_TRY(check_rows(v + 8, 5, esz));
    }
    GDN_TRY(check_alignment(v + 1, 7, 4));
    GDN_TRY(check_overlap(v, kSsmViews, 2));
    gdn_record_launch(0, -1);
    *nothing = a.N == 0 || (rows == 0 && !a.state_out);
    if (!a.state_in && !a.state_out) a.slots = nullptr;  // no pool that a slot could be past the end of
    return GDN_OK;
}

size_t align16(size_t x) { return (x + 15) & ~(size_t)15; }

size_t ssm_workspace(int64_t slots, int channels, int d_state)
{
    return align16((size_t)slots * channels * d_state * 4) + align16((size_t)slots * channels * 4);
}

// Cuts the call into pieces if it is to be, and lays out the workspace.
gdn_status_t take_workspace(GdnSsmArgs &a, int asked, void *workspace, size_t bytes)
{
    gdn_ssm_plan(a.N, a.T, a.channels, a.groups, a.cu_seqlens != nullptr, asked, &a.segment, &a.pieces);
    if (!a.segment) return GDN_OK;
    const size_t need = ssm_workspace(a.pieces, a.channels, a.d_state);
    if (!workspace || bytes < need)
        return gdn_fail(GDN_ERR_INVALID_ARG, "workspace of %zu bytes needed (%zu given)", need,
                        workspace ? bytes : (size_t)0);
    View v[kSsmViews + 1];
    v[0] = flat("workspace", workspace, need);
    GDN_TRY(check_alignment(v, 1, 16));
    ssm_views(a, a.cu_seqlens ? a.T : (int64_t)a.N * a.T, v + 1);
    GDN_TRY(check_overlap(v, kSsmViews + 1, 1));
    a.piece_state = static_cast<float *>(workspace);
    a.piece_delta = a.piece_state + align16((size_t)a.pieces * a.channels * a.d_state * 4) / 4;
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status_t gdn_conv_fwd(const void *x, const float *weight, const float *bias,
                          const void *state_in, const int32_t *slots, void *y, void *state_out,
                          int B, int T, int channels, int width, int64_t ld_x, int64_t ld_y,
                          int pool, const int32_t *cu_seqlens, gdn_act_t act, gdn_dtype_t dtype,
                          void *stream)
{
    GdnConvArgs a = {x, weight, bias, state_in, slots, y, state_out, B, T, channels, width,
                     ld_x, ld_y, pool, cu_seqlens, 0, 0, nullptr};
    return conv(false, a, act, dtype, stream);
}

gdn_status_t gdn_conv_step(const void *x, const float *weight, const float *bias,
                           const void *state_in, const int32_t *slots, void *y, void *state_out,
                           int N, int channels, int width, int64_t ld_x, int64_t ld_y, int pool,
                           gdn_act_t act, gdn_dtype_t dtype, void *stream)
{
    GdnConvArgs a = {x, weight, bias, state_in, slots, y, state_out, N, 1, channels, width,
                     ld_x, ld_y, pool, nullptr, 0, 0, nullptr};
    return conv(true, a, act, dtype, stream);
}

size_t gdn_ssm_fwd_workspace_size(int B, int T, int channels, int d_state,
                                  const int32_t *cu_seqlens, int segment)
{
    if (B < 1 || T < 1 || channels < 1 || d_state < 1 || d_state > 128) return 0;
    int seg = 0;
    int64_t slots = 0;
    gdn_ssm_plan(B, T, channels, 1, cu_seqlens != nullptr, segment, &seg, &slots);  // enough for any groups
    return seg ? ssm_workspace(slots, channels, d_state) : 0;
}

gdn_status_t gdn_ssm_fwd(const void *x, const void *delta, const float *A, const void *Bm,
                         const void *Cm, const float *D, const void *z, const float *delta_bias,
                         const float *state_in, const int32_t *slots, void *y, float *state_out,
                         int B, int T, int channels, int d_state, int groups, int64_t ld_x,
                         int64_t ld_delta, int64_t ld_b, int64_t ld_c, int64_t ld_z, int64_t ld_y,
                         int pool, const int32_t *cu_seqlens, int delta_softplus,
                         gdn_dtype_t dtype, int segment, void *workspace, size_t workspace_bytes,
                         void *stream)
{
    GdnSsmArgs a = {x, delta, Bm, Cm, z, A, D, delta_bias, state_in, slots, y, state_out, B, T,
                    channels, d_state, groups, ld_x, ld_delta, ld_b, ld_c, ld_z, ld_y, pool,
                    cu_seqlens, delta_softplus};
    bool nothing = false;
    GDN_TRY(check_ssm(false, a, dtype, &nothing));
    if (nothing) return GDN_OK;
    if (T > 0) GDN_TRY(take_workspace(a, segment, workspace, workspace_bytes));
    GDN_TRY(gdn_device_status_word(&a.status));
    int launches = 0;
    const cudaError_t e = gdn_launch_ssm_fwd(a, static_cast<cudaStream_t>(stream), &launches);
    return launched(e, "state space scan", launches, 7);
}

gdn_status_t gdn_ssm_step(const void *x, const void *delta, const float *A, const void *Bm,
                          const void *Cm, const float *D, const void *z, const float *delta_bias,
                          const float *state_in, const int32_t *slots, void *y, float *state_out,
                          int N, int channels, int d_state, int groups, int64_t ld_x,
                          int64_t ld_delta, int64_t ld_b, int64_t ld_c, int64_t ld_z, int64_t ld_y,
                          int pool, int delta_softplus, gdn_dtype_t dtype, void *stream)
{
    GdnSsmArgs a = {x, delta, Bm, Cm, z, A, D, delta_bias, state_in, slots, y, state_out, N, 1,
                    channels, d_state, groups, ld_x, ld_delta, ld_b, ld_c, ld_z, ld_y, pool,
                    nullptr, delta_softplus};
    bool nothing = false;
    GDN_TRY(check_ssm(true, a, dtype, &nothing));
    if (nothing) return GDN_OK;
    GDN_TRY(gdn_device_status_word(&a.status));
    return launched(gdn_launch_ssm_step(a, static_cast<cudaStream_t>(stream)), "state space step", 1, 7);
}

gdn_status_t gdn_group_norm(const void *x, const void *gate, const float *weight,
                            const float *bias, void *y, int64_t rows, int channels, int groups,
                            int64_t ld_x, int64_t ld_gate, int64_t ld_y, float eps, int rms,
                            gdn_act_t act, gdn_dtype_t dtype, void *stream)
{
    gdn_begin_call();
    if (rows < 0) return gdn_fail(GDN_ERR_INVALID_ARG, "negative size: %lld rows", (long long)rows);
    if (channels < 1 || groups < 1 || channels % groups)
        return gdn_fail(GDN_ERR_INVALID_ARG, "%d channels are not a multiple of %d groups", channels, groups);
    if (!(eps >= 0.f)) return gdn_fail(GDN_ERR_INVALID_ARG, "eps must be >= 0: %g", (double)eps);
    GDN_TRY(check_types(dtype, act));
    if (rows > 0 && (!x || !y)) return gdn_fail(GDN_ERR_INVALID_ARG, "x and y must be non-NULL");
    const size_t esz = dtype == GDN_BF16 ? 2 : 4, row = (size_t)channels * esz;
    View v[] = {{"y", y, rows, row, (size_t)ld_y * esz},
                {"x", x, rows, row, (size_t)ld_x * esz},
                {"gate", gate, rows, row, (size_t)ld_gate * esz},
                flat("weight", weight, (size_t)channels * 4),
                flat("bias", bias, (size_t)channels * 4)};
    if (rows > 0) GDN_TRY(check_rows(v, 3, esz));
    GDN_TRY(check_alignment(v + 3, 2, 4));
    if (y == x && (ld_y == ld_x || rows == 1)) v[1].p = nullptr;  // in place
    if (y == gate && (ld_y == ld_gate || rows == 1)) v[2].p = nullptr;
    GDN_TRY(check_overlap(v, 5, 1));
    gdn_record_launch(0, -1);
    if (rows == 0) return GDN_OK;
    GdnNormArgs a = {x, gate, weight, bias, y, rows, channels, groups, ld_x, ld_gate, ld_y, eps, rms,
                     act, dtype == GDN_BF16 ? 1 : 0};
    return launched(gdn_launch_group_norm(a, static_cast<cudaStream_t>(stream)), "group norm", 1, 8);
}

}  // extern "C"
