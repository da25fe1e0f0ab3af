// abi.hip -- the C ABI (include/ssm_mi355x.h): argument checks, path selection, launches.
// Host code only; every computation runs in the kernels of conv.hip, recurrent.hip and
// ssd.hip.  Nothing here allocates device memory, synchronises, throws or prints.
#include <cmath>
#include <mutex>
#include <string>
#include <utility>
#include <vector>

#include "delta.h"
#include "internal.h"

namespace {

thread_local std::string g_err;

ssm_status_t fail(ssm_status_t s, const std::string& msg) {
    g_err = msg;
    return s;
}
ssm_status_t ok() {
    g_err.clear();
    return SSM_OK;
}
ssm_status_t hip_status(hipError_t e, const char* where) {
    if (e == hipSuccess) return ok();
    g_err = std::string(where) + ": " + hipGetErrorString(e);
    return SSM_ERR_HIP;
}
size_t esize(ssm_dtype_t d) { return d == SSM_BF16 ? 2 : 4; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool valid_dtype(int d) { return d == SSM_F32 || d == SSM_BF16; }
bool valid_act(int a) { return a == SSM_ACT_NONE || a == SSM_ACT_SILU; }

// ---- optional kernel timing (measurement only) ----
std::mutex g_tmu;
bool g_timing = false;
struct EventPair {
    hipEvent_t e0, e1;
    int dev;
};
std::vector<EventPair> g_events;  // recorded, not yet read
std::vector<EventPair> g_spare;   // read, kept for reuse (created once, never per launch)

// Pointer arguments: name, pointer, required?, element alignment.
struct PtrCheck {
    const char* name;
    const void* p;
    bool required;
    size_t align;
};
ssm_status_t check_ptrs(const char* fn, std::initializer_list<PtrCheck> list) {
    for (const auto& c : list) {
        if (c.p == nullptr) {
            if (c.required) return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": " + c.name + " is NULL");
            continue;
        }
        if (!aligned(c.p, c.align))
            return fail(SSM_ERR_ALIGNMENT, std::string(fn) + ": " + c.name + " is not aligned to " +
                                               std::to_string(c.align) + " bytes");
    }
    return SSM_OK;
}

ssm_status_t check_scan_dims(const char* fn, int64_t batch, int64_t seqlen, int64_t nheads,
                             int64_t headdim, int64_t ngroups, int64_t dstate, int dtype) {
    if (!valid_dtype(dtype)) return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": bad dtype");
    if (batch < 0 || seqlen < 0)
        return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": negative batch or seqlen");
    if (nheads < 1 || headdim < 1 || ngroups < 1 || dstate < 1)
        return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": nheads, headdim, ngroups, dstate must be >= 1");
    if (nheads % ngroups != 0)
        return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": nheads is not a multiple of ngroups");
    return SSM_OK;
}

}  // namespace

extern "C" {

int ssm_abi_version(void) { return SSM_ABI_VERSION; }

const char* ssm_status_string(int32_t s) {
    switch (s) {
        case SSM_OK: return "ok";
        case SSM_ERR_INVALID_ARG: return "invalid argument";
        case SSM_ERR_UNSUPPORTED: return "unsupported sizes or dtype";
        case SSM_ERR_ALIGNMENT: return "misaligned pointer";
        case SSM_ERR_WORKSPACE: return "workspace missing or too small";
        case SSM_ERR_HIP: return "HIP runtime error";
    }
    return "unknown status";
}

const char* ssm_last_error(void) { return g_err.c_str(); }

ssm_status_t ssm_conv1d_fwd(const void* x, const float* w, const float* bias,
                            const void* initial_state, void* final_state,
                            const int32_t* seq_idx, void* out, int64_t batch, int64_t seqlen,
                            int64_t channels, int64_t width, ssm_dtype_t dtype, ssm_act_t act,
                            ssm_stream_t stream) {
    const char* fn = "ssm_conv1d_fwd";
    if (!valid_dtype(dtype)) return fail(SSM_ERR_INVALID_ARG, "ssm_conv1d_fwd: bad dtype");
    if (!valid_act(act)) return fail(SSM_ERR_INVALID_ARG, "ssm_conv1d_fwd: bad activation");
    if (batch < 0 || seqlen < 0 || channels < 1)
        return fail(SSM_ERR_INVALID_ARG, "ssm_conv1d_fwd: need batch >= 0, seqlen >= 0, channels >= 1");
    if (width < 2 || width > 8)
        return fail(SSM_ERR_UNSUPPORTED, "ssm_conv1d_fwd: width must be in [2, 8]");
    const size_t es = esize(dtype);
    const bool work = batch > 0 && seqlen > 0;
    ssm_status_t st = check_ptrs(fn, {{"x", x, work, es},
                                      {"w", w, work, 4},
                                      {"bias", bias, false, 4},
                                      {"initial_state", initial_state, false, es},
                                      {"final_state", final_state, false, es},
                                      {"seq_idx", seq_idx, false, 4},
                                      {"out", out, work, es}});
    if (st != SSM_OK) return st;
    if (batch == 0) return ok();
    return hip_status(ssm::launch_conv1d_fwd(x, w, bias, initial_state, final_state, seq_idx, out,
                                             batch, seqlen, channels, width, dtype, act,
                                             reinterpret_cast<hipStream_t>(stream)),
                      fn);
}

ssm_status_t ssm_conv1d_update(const void* x, void* conv_state, const float* w,
                               const float* bias, const int32_t* conv_state_indices,
                               const int32_t* cache_seqlens, void* out, int64_t batch,
                               int64_t channels, int64_t n_new, int64_t width,
                               int64_t state_len, int64_t n_slots, ssm_dtype_t dtype,
                               ssm_act_t act, ssm_stream_t stream) {
    const char* fn = "ssm_conv1d_update";
    if (!valid_dtype(dtype)) return fail(SSM_ERR_INVALID_ARG, "ssm_conv1d_update: bad dtype");
    if (!valid_act(act)) return fail(SSM_ERR_INVALID_ARG, "ssm_conv1d_update: bad activation");
    if (batch < 0 || n_new < 0 || channels < 1 || n_slots < 1)
        return fail(SSM_ERR_INVALID_ARG,
                    "ssm_conv1d_update: need batch >= 0, n_new >= 0, channels >= 1, n_slots >= 1");
    if (width < 2 || width > 8)
        return fail(SSM_ERR_UNSUPPORTED, "ssm_conv1d_update: width must be in [2, 8]");
    if (state_len < width - 1)
        return fail(SSM_ERR_INVALID_ARG, "ssm_conv1d_update: state_len < width - 1");
    const size_t es = esize(dtype);
    const bool work = batch > 0 && n_new > 0;
    ssm_status_t st = check_ptrs(fn, {{"x", x, work, es},
                                      {"conv_state", conv_state, work, es},
                                      {"w", w, work, 4},
                                      {"bias", bias, false, 4},
                                      {"conv_state_indices", conv_state_indices, false, 4},
                                      {"cache_seqlens", cache_seqlens, false, 4},
                                      {"out", out, work, es}});
    if (st != SSM_OK) return st;
    if (!work) return ok();
    return hip_status(ssm::launch_conv1d_update(x, conv_state, w, bias, conv_state_indices,
                                                cache_seqlens, out, batch, channels, n_new, width,
                                                state_len, n_slots, dtype, act,
                                                reinterpret_cast<hipStream_t>(stream)),
                      fn);
}

size_t ssm_scan_workspace_size(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                               int64_t ngroups, int64_t dstate, ssm_dtype_t dtype) {
    if (batch <= 0 || seqlen <= 0 || nheads < 1 || headdim < 1 || ngroups < 1 || dstate < 1 ||
        !valid_dtype(dtype))
        return 0;
    if (ssm::chunked_supported(headdim, dstate, dtype))
        return ssm::chunked_workspace_bytes(batch, seqlen, nheads, ngroups, dstate);
    // general-shape path of the fused call: the conv output is staged in the workspace
    return static_cast<size_t>(batch * seqlen * (nheads * headdim + 2 * ngroups * dstate)) *
           esize(dtype);
}

namespace {

// Shared tail of ssm_scan_fwd / ssm_conv_scan_fwd on the token-sequential path.
ssm_status_t run_recurrent_scan(const char* fn, const void* x, int64_t x_row, const void* Bm,
                                const void* Cm, int64_t bc_row, const float* dt, const float* A,
                                const float* initial_state, float* final_state,
                                const int32_t* seq_idx, void* y, int64_t batch, int64_t seqlen,
                                int64_t nheads, int64_t headdim, int64_t ngroups,
                                int64_t dstate, ssm_dtype_t dtype, hipStream_t s) {
    ssm::RecurrentArgs r{};
    r.x = x;
    r.x_sb = seqlen * x_row;
    r.x_st = x_row;
    r.x_sc = 1;
    r.dt = dt;
    r.A = A;
    r.Bm = Bm;
    r.B_sb = seqlen * bc_row;
    r.B_st = bc_row;
    r.B_sc = 1;
    r.Cm = Cm;
    r.C_sb = seqlen * bc_row;
    r.C_st = bc_row;
    r.C_sc = 1;
    r.state_in = initial_state;
    r.state_out = final_state;
    r.indices = nullptr;
    r.n_slots = batch;
    r.seq_idx = seq_idx;
    r.y = y;
    r.B = batch;
    r.T = seqlen;
    r.H = nheads;
    r.P = headdim;
    r.G = ngroups;
    r.N = dstate;
    return hip_status(ssm::launch_recurrent(r, dtype, s), fn);
}

hipEvent_t g_none = nullptr;

// Events for the timing record (both NULL when timing is off): a pair from the spare list
// of the current device when there is one, else a new pair (created once; ssm_timing_read
// returns pairs to the spare list instead of destroying them).
ssm_status_t timing_events(hipEvent_t* ev0, hipEvent_t* ev1) {
    *ev0 = *ev1 = g_none;
    std::lock_guard<std::mutex> lk(g_tmu);
    if (!g_timing) return SSM_OK;
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_status(e, "timing");
    for (size_t i = g_spare.size(); i-- > 0;) {
        if (g_spare[i].dev == dev) {
            g_events.push_back(g_spare[i]);
            g_spare.erase(g_spare.begin() + static_cast<std::ptrdiff_t>(i));
            *ev0 = g_events.back().e0;
            *ev1 = g_events.back().e1;
            return SSM_OK;
        }
    }
    e = hipEventCreate(ev0);
    if (e == hipSuccess) e = hipEventCreate(ev1);
    if (e != hipSuccess) return hip_status(e, "timing");
    g_events.push_back({*ev0, *ev1, dev});
    return SSM_OK;
}

}  // namespace

ssm_status_t ssm_scan_fwd(const void* x, const float* dt, const float* A, const void* Bm,
                          const void* Cm, const float* initial_state, float* final_state,
                          const int32_t* seq_idx, void* y, int64_t batch, int64_t seqlen,
                          int64_t nheads, int64_t headdim, int64_t ngroups, int64_t dstate,
                          ssm_dtype_t dtype, void* workspace, size_t workspace_bytes,
                          ssm_stream_t stream) {
    const char* fn = "ssm_scan_fwd";
    ssm_status_t st = check_scan_dims(fn, batch, seqlen, nheads, headdim, ngroups, dstate, dtype);
    if (st != SSM_OK) return st;
    const size_t es = esize(dtype);
    const bool work = batch > 0 && seqlen > 0;
    st = check_ptrs(fn, {{"x", x, work, es},
                         {"dt", dt, work, 4},
                         {"A", A, work, 4},
                         {"Bm", Bm, work, es},
                         {"Cm", Cm, work, es},
                         {"initial_state", initial_state, false, 16},
                         {"final_state", final_state, false, 16},
                         {"seq_idx", seq_idx, false, 4},
                         {"y", y, work, es}});
    if (st != SSM_OK) return st;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (batch == 0) return ok();
    if (seqlen == 0)
        return hip_status(ssm::launch_copy_or_zero_f32(final_state, initial_state,
                                                       batch * nheads * headdim * dstate, s),
                          fn);
    // the matrix-core path loads x, Bm and Cm rows in 16-byte pieces and stores y in 8-byte
    // pieces; other alignments take the token-sequential path
    if (ssm::chunked_supported(headdim, dstate, dtype) && aligned(x, 16) && aligned(Bm, 16) &&
        aligned(Cm, 16) && aligned(y, 8)) {
        const size_t need = ssm::chunked_workspace_bytes(batch, seqlen, nheads, ngroups, dstate);
        if (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16))
            return fail(SSM_ERR_WORKSPACE, "ssm_scan_fwd: workspace must be >= " +
                                               std::to_string(need) + " bytes, 16-byte aligned");
        ssm::ChunkedArgs a{};
        a.x = static_cast<const uint16_t*>(x);
        a.x_row = nheads * headdim;
        a.x_col0 = 0;
        a.bsrc = static_cast<const uint16_t*>(Bm);
        a.b_row = ngroups * dstate;
        a.b_col0 = 0;
        a.csrc = static_cast<const uint16_t*>(Cm);
        a.c_row = ngroups * dstate;
        a.c_col0 = 0;
        a.fused_conv = false;
        a.K = 2;  // no conv: one halo row staged and ignored
        a.C_conv = 0;
        a.act = SSM_ACT_NONE;
        a.dt = dt;
        a.A = A;
        a.init_state = initial_state;
        a.final_state = final_state;
        a.seq_idx = seq_idx;
        a.y = static_cast<uint16_t*>(y);
        a.B = batch;
        a.L = seqlen;
        a.H = nheads;
        a.P = headdim;
        a.G = ngroups;
        a.N = dstate;
        a.workspace = workspace;
        hipEvent_t e0, e1;
        st = timing_events(&e0, &e1);
        if (st != SSM_OK) return st;
        return hip_status(ssm::launch_chunked(a, s, e0, e1), fn);
    }
    if (!ssm::recurrent_supported(headdim, dstate))
        return fail(SSM_ERR_UNSUPPORTED, "ssm_scan_fwd: dstate must be 4 * 2^k <= 256 and headdim*dstate <= 16384");
    return run_recurrent_scan(fn, x, nheads * headdim, Bm, Cm, ngroups * dstate, dt, A,
                              initial_state, final_state, seq_idx, y, batch, seqlen, nheads,
                              headdim, ngroups, dstate, dtype, s);
}

namespace {

// Body of ssm_conv_scan_fwd and ssm_conv_scan_fwd_noalloc; `timed` lets the main-kernel
// timing record (when switched on) create its events.
ssm_status_t conv_scan_fwd_impl(const char* fn, const void* xBC, const float* conv_w,
                                const float* conv_bias, const void* conv_initial_state,
                                void* conv_final_state, const float* dt, const float* A,
                                const float* initial_state, float* final_state,
                                const int32_t* seq_idx, void* y, int64_t batch, int64_t seqlen,
                                int64_t nheads, int64_t headdim, int64_t ngroups, int64_t dstate,
                                int64_t width, ssm_dtype_t dtype, ssm_act_t act, void* workspace,
                                size_t workspace_bytes, bool timed, ssm_stream_t stream,
                                const int32_t* state_slots = nullptr, int64_t n_state_slots = 0) {
    // n_state_slots > 0 (the pooled prefill, chunked shapes only): the SSM states are rows
    // state_slots[b] of an [n_state_slots, H, P, N] pool, read and written in place
    ssm_status_t st = check_scan_dims(fn, batch, seqlen, nheads, headdim, ngroups, dstate, dtype);
    if (st != SSM_OK) return st;
    if (!valid_act(act)) return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": bad activation");
    if (width < 2 || width > 8)
        return fail(SSM_ERR_UNSUPPORTED, std::string(fn) + ": width must be in [2, 8]");
    const size_t es = esize(dtype);
    const bool work = batch > 0 && seqlen > 0;
    st = check_ptrs(fn, {{"xBC", xBC, work, es},
                         {"conv_w", conv_w, work, 4},
                         {"conv_bias", conv_bias, false, 4},
                         {"conv_initial_state", conv_initial_state, false, es},
                         {"conv_final_state", conv_final_state, false, es},
                         {"dt", dt, work, 4},
                         {"A", A, work, 4},
                         {"initial_state", initial_state, false, 16},
                         {"final_state", final_state, false, 16},
                         {"seq_idx", seq_idx, false, 4},
                         {"y", y, work, es}});
    if (st != SSM_OK) return st;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const int64_t C_conv = nheads * headdim + 2 * ngroups * dstate;
    if (batch == 0) return ok();
    if (seqlen == 0) {
        hipError_t e = ssm::launch_conv1d_fwd(nullptr, conv_w, conv_bias, conv_initial_state,
                                              conv_final_state, nullptr, nullptr, batch, 0,
                                              C_conv, width, dtype, act, s);
        // pool rows stay where they are: nothing to copy
        if (e == hipSuccess && n_state_slots <= 0)
            e = ssm::launch_copy_or_zero_f32(final_state, initial_state,
                                             batch * nheads * headdim * dstate, s);
        return hip_status(e, fn);
    }
    if (ssm::chunked_supported(headdim, dstate, dtype)) {
        const size_t need = ssm::chunked_workspace_bytes(batch, seqlen, nheads, ngroups, dstate);
        if (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16))
            return fail(SSM_ERR_WORKSPACE, std::string(fn) + ": workspace must be >= " +
                                               std::to_string(need) + " bytes, 16-byte aligned");
        if (!aligned(xBC, 16) || C_conv % 8 != 0 || !aligned(y, 8))
            return fail(SSM_ERR_ALIGNMENT,
                        std::string(fn) + ": xBC must be 16-byte aligned with a channel count "
                        "divisible by 8, y 8-byte aligned");
        ssm::ChunkedArgs a{};
        a.x = static_cast<const uint16_t*>(xBC);
        a.x_row = C_conv;
        a.x_col0 = 0;
        a.bsrc = a.x;
        a.b_row = C_conv;
        a.b_col0 = nheads * headdim;
        a.csrc = a.x;
        a.c_row = C_conv;
        a.c_col0 = nheads * headdim + ngroups * dstate;
        a.fused_conv = true;
        a.conv_w = conv_w;
        a.conv_b = conv_bias;
        a.conv_init = static_cast<const uint16_t*>(conv_initial_state);
        a.conv_final = static_cast<uint16_t*>(conv_final_state);
        a.C_conv = C_conv;
        a.K = width;
        a.act = act;
        a.dt = dt;
        a.A = A;
        a.init_state = initial_state;
        a.final_state = final_state;
        a.state_slots = state_slots;
        a.n_state_slots = n_state_slots;
        a.seq_idx = seq_idx;
        a.y = static_cast<uint16_t*>(y);
        a.B = batch;
        a.L = seqlen;
        a.H = nheads;
        a.P = headdim;
        a.G = ngroups;
        a.N = dstate;
        a.workspace = workspace;
        hipEvent_t e0 = g_none, e1 = g_none;
        if (timed) {
            st = timing_events(&e0, &e1);
            if (st != SSM_OK) return st;
        }
        return hip_status(ssm::launch_chunked(a, s, e0, e1), fn);
    }
    // general shapes: conv into the workspace, then the token-sequential scan reading its
    // x | B | C channel ranges in place
    if (n_state_slots > 0)
        return fail(SSM_ERR_UNSUPPORTED, std::string(fn) + ": pool rows need the chunked path");
    if (!ssm::recurrent_supported(headdim, dstate))
        return fail(SSM_ERR_UNSUPPORTED, std::string(fn) + ": dstate must be 4 * 2^k <= 256 and headdim*dstate <= 16384");
    const size_t need = static_cast<size_t>(batch * seqlen * C_conv) * es;
    if (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16))
        return fail(SSM_ERR_WORKSPACE, std::string(fn) + ": workspace must be >= " +
                                           std::to_string(need) + " bytes, 16-byte aligned");
    hipError_t e = ssm::launch_conv1d_fwd(xBC, conv_w, conv_bias, conv_initial_state,
                                          conv_final_state, seq_idx, workspace, batch, seqlen,
                                          C_conv, width, dtype, act, s);
    if (e != hipSuccess) return hip_status(e, fn);
    const uint8_t* base = static_cast<const uint8_t*>(workspace);
    return run_recurrent_scan(fn, base, C_conv, base + nheads * headdim * es,
                              base + (nheads * headdim + ngroups * dstate) * es, C_conv, dt, A,
                              initial_state, final_state, seq_idx, y, batch, seqlen, nheads,
                              headdim, ngroups, dstate, dtype, s);
}

}  // namespace

ssm_status_t ssm_conv_scan_fwd(const void* xBC, const float* conv_w, const float* conv_bias,
                               const void* conv_initial_state, void* conv_final_state,
                               const float* dt, const float* A, const float* initial_state,
                               float* final_state, const int32_t* seq_idx, void* y,
                               int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                               int64_t ngroups, int64_t dstate, int64_t width,
                               ssm_dtype_t dtype, ssm_act_t act, void* workspace,
                               size_t workspace_bytes, ssm_stream_t stream) {
    return conv_scan_fwd_impl("ssm_conv_scan_fwd", xBC, conv_w, conv_bias, conv_initial_state,
                              conv_final_state, dt, A, initial_state, final_state, seq_idx, y,
                              batch, seqlen, nheads, headdim, ngroups, dstate, width, dtype, act,
                              workspace, workspace_bytes, true, stream);
}

// ---------------------------------------------------------------------------------------
// Allocation-free fused prefill: the workspace is a static device array of the library.
// ---------------------------------------------------------------------------------------
namespace {

constexpr size_t kScratchBytes = size_t(32) << 20;
constexpr int kMaxDevices = 64;

// One copy per GPU, created when the library's code object is loaded on that GPU and held
// until the process ends.  Host code never passes `scratch` itself to a kernel (its host-side
// name is not a device address); it uses the per-device address from scratch_address().
static __device__ __align__(256) uint8_t scratch[kScratchBytes];

std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

// Device address of the current device's scratch, looked up once per device.
ssm_status_t scratch_address(const char* fn, void** out) {
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_status(e, fn);
    if (dev < 0 || dev >= kMaxDevices)
        return fail(SSM_ERR_UNSUPPORTED, std::string(fn) + ": device ordinal " +
                                             std::to_string(dev) + " beyond the scratch table");
    std::lock_guard<std::mutex> lk(g_scratch_mu);
    if (g_scratch_ptr[dev] == nullptr) {
        void* p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (e != hipSuccess) return hip_status(e, fn);
        if (p == nullptr) return fail(SSM_ERR_HIP, std::string(fn) + ": scratch has no address");
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return SSM_OK;
}

}  // namespace

size_t ssm_noalloc_scratch_bytes(void) { return kScratchBytes; }

ssm_status_t ssm_conv_scan_fwd_noalloc(const void* xBC, const float* conv_w,
                                       const float* conv_bias, const void* conv_initial_state,
                                       void* conv_final_state, const float* dt, const float* A,
                                       const float* initial_state, float* final_state,
                                       const int32_t* seq_idx, void* y, int64_t batch,
                                       int64_t seqlen, int64_t nheads, int64_t headdim,
                                       int64_t ngroups, int64_t dstate, int64_t width,
                                       ssm_dtype_t dtype, ssm_act_t act, ssm_stream_t stream) {
    const char* fn = "ssm_conv_scan_fwd_noalloc";
    const size_t need = ssm_scan_workspace_size(batch, seqlen, nheads, headdim, ngroups, dstate,
                                                dtype);
    if (need > kScratchBytes)
        return fail(SSM_ERR_WORKSPACE, std::string(fn) + ": these sizes need " +
                                           std::to_string(need) + " bytes of scratch; the static "
                                           "scratch holds " + std::to_string(kScratchBytes) +
                                           " (ssm_conv_scan_fwd takes a workspace of any size)");
    void* ws = nullptr;
    if (batch > 0 && seqlen > 0) {
        // argument errors are reported before the scratch is looked up
        ssm_status_t st = check_scan_dims(fn, batch, seqlen, nheads, headdim, ngroups, dstate,
                                          dtype);
        if (st != SSM_OK) return st;
        st = scratch_address(fn, &ws);
        if (st != SSM_OK) return st;
    }
    return conv_scan_fwd_impl(fn, xBC, conv_w, conv_bias, conv_initial_state, conv_final_state,
                              dt, A, initial_state, final_state, seq_idx, y, batch, seqlen,
                              nheads, headdim, ngroups, dstate, width, dtype, act, ws,
                              ws ? kScratchBytes : 0, false, stream);
}

ssm_status_t ssm_step(const void* x, int64_t x_sb, int64_t x_st, int64_t x_sc, const float* dt,
                      const float* A, const void* Bm, int64_t B_sb, int64_t B_st, int64_t B_sc,
                      const void* Cm, int64_t C_sb, int64_t C_st, int64_t C_sc, float* state,
                      const int32_t* state_indices, void* y, int64_t batch, int64_t n_new,
                      int64_t nheads, int64_t headdim, int64_t ngroups, int64_t dstate,
                      int64_t n_slots, ssm_dtype_t dtype, ssm_stream_t stream) {
    const char* fn = "ssm_step";
    ssm_status_t st = check_scan_dims(fn, batch, n_new, nheads, headdim, ngroups, dstate, dtype);
    if (st != SSM_OK) return st;
    if (n_slots < 1) return fail(SSM_ERR_INVALID_ARG, "ssm_step: n_slots must be >= 1");
    if (!ssm::recurrent_supported(headdim, dstate))
        return fail(SSM_ERR_UNSUPPORTED, "ssm_step: dstate must be 4 * 2^k <= 256 and headdim*dstate <= 16384");
    const size_t es = esize(dtype);
    const bool work = batch > 0 && n_new > 0;
    st = check_ptrs(fn, {{"x", x, work, es},
                         {"dt", dt, work, 4},
                         {"A", A, work, 4},
                         {"Bm", Bm, work, es},
                         {"Cm", Cm, work, es},
                         {"state", state, work, 16},
                         {"state_indices", state_indices, false, 4},
                         {"y", y, work, es}});
    if (st != SSM_OK) return st;
    if (!work) return ok();
    ssm::RecurrentArgs r{};
    r.x = x;
    r.x_sb = x_sb;
    r.x_st = x_st;
    r.x_sc = x_sc;
    r.dt = dt;
    r.A = A;
    r.Bm = Bm;
    r.B_sb = B_sb;
    r.B_st = B_st;
    r.B_sc = B_sc;
    r.Cm = Cm;
    r.C_sb = C_sb;
    r.C_st = C_st;
    r.C_sc = C_sc;
    r.state_in = state;
    r.state_out = state;
    r.indices = state_indices;
    r.n_slots = n_slots;
    r.seq_idx = nullptr;
    r.y = y;
    r.B = batch;
    r.T = n_new;
    r.H = nheads;
    r.P = headdim;
    r.G = ngroups;
    r.N = dstate;
    return hip_status(ssm::launch_recurrent(r, dtype, reinterpret_cast<hipStream_t>(stream)), fn);
}

ssm_status_t ssm_decode_step(const void* x_new, void* conv_state, const float* conv_w,
                             const float* conv_bias, const int32_t* conv_state_indices,
                             const int32_t* cache_seqlens, const float* dt, const float* A,
                             float* ssm_state, const int32_t* state_indices, void* conv_out,
                             void* y, int64_t batch, int64_t n_new, int64_t nheads,
                             int64_t headdim, int64_t ngroups, int64_t dstate, int64_t width,
                             int64_t state_len, int64_t n_conv_slots, int64_t n_ssm_slots,
                             ssm_dtype_t dtype, ssm_act_t act, ssm_stream_t stream) {
    const char* fn = "ssm_decode_step";
    ssm_status_t st = check_scan_dims(fn, batch, n_new, nheads, headdim, ngroups, dstate, dtype);
    if (st != SSM_OK) return st;
    if (!valid_act(act)) return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": bad activation");
    if (n_conv_slots < 1 || n_ssm_slots < 1)
        return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": n_conv_slots and n_ssm_slots must be >= 1");
    if (width < 2 || width > 8)
        return fail(SSM_ERR_UNSUPPORTED, std::string(fn) + ": width must be in [2, 8]");
    if (state_len < width - 1)
        return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": state_len < width - 1");
    if (!ssm::recurrent_supported(headdim, dstate))
        return fail(SSM_ERR_UNSUPPORTED, std::string(fn) + ": dstate must be 4 * 2^k <= 256 and headdim*dstate <= 16384");
    const size_t es = esize(dtype);
    const bool work = batch > 0 && n_new > 0;
    st = check_ptrs(fn, {{"x_new", x_new, work, es},
                         {"conv_state", conv_state, work, es},
                         {"conv_w", conv_w, work, 4},
                         {"conv_bias", conv_bias, false, 4},
                         {"conv_state_indices", conv_state_indices, false, 4},
                         {"cache_seqlens", cache_seqlens, false, 4},
                         {"dt", dt, work, 4},
                         {"A", A, work, 4},
                         {"ssm_state", ssm_state, work, 16},
                         {"state_indices", state_indices, false, 4},
                         {"conv_out", conv_out, work, es},
                         {"y", y, work, es}});
    if (st != SSM_OK) return st;
    if (!work) return ok();
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const int64_t C = nheads * headdim + 2 * ngroups * dstate;
    const int64_t HP = nheads * headdim, GN = ngroups * dstate;
    ssm::RecurrentArgs r{};
    r.x = conv_out;  // x | B | C channel ranges of the conv output [batch, C, n_new]
    r.x_sb = C * n_new;
    r.x_st = 1;
    r.x_sc = n_new;
    r.dt = dt;
    r.A = A;
    r.Bm = static_cast<const uint8_t*>(conv_out) + HP * n_new * es;
    r.B_sb = C * n_new;
    r.B_st = 1;
    r.B_sc = n_new;
    r.Cm = static_cast<const uint8_t*>(conv_out) + (HP + GN) * n_new * es;
    r.C_sb = C * n_new;
    r.C_st = 1;
    r.C_sc = n_new;
    r.state_in = ssm_state;
    r.state_out = ssm_state;
    r.indices = state_indices ? state_indices : conv_state_indices;
    r.n_slots = n_ssm_slots;
    r.seq_idx = nullptr;
    r.y = y;
    r.B = batch;
    r.T = n_new;
    r.H = nheads;
    r.P = headdim;
    r.G = ngroups;
    r.N = dstate;
    hipError_t e = ssm::launch_conv1d_update(x_new, conv_state, conv_w, conv_bias,
                                             conv_state_indices, cache_seqlens, conv_out, batch,
                                             C, n_new, width, state_len, n_conv_slots, dtype, act,
                                             s);
    if (e != hipSuccess) return hip_status(e, fn);
    return hip_status(ssm::launch_recurrent(r, dtype, s), fn);
}

ssm_status_t ssm_scan_fwd_vector_decay(const void* x, const float* dt, const float* log_decay,
                                       const float* A_vec, const void* Bm, const void* Cm,
                                       const float* initial_state, float* final_state,
                                       const int32_t* seq_idx, void* y, int64_t batch,
                                       int64_t seqlen, int64_t nheads, int64_t headdim,
                                       int64_t ngroups, int64_t dstate, ssm_dtype_t dtype,
                                       ssm_stream_t stream) {
    const char* fn = "ssm_scan_fwd_vector_decay";
    ssm_status_t st = check_scan_dims(fn, batch, seqlen, nheads, headdim, ngroups, dstate, dtype);
    if (st != SSM_OK) return st;
    const size_t es = esize(dtype);
    const bool rows = batch > 0;
    const bool work = rows && seqlen > 0;
    // the decay source matters only when there are tokens (an empty tensor has no address)
    if (work && (log_decay == nullptr) == (A_vec == nullptr))
        return fail(SSM_ERR_INVALID_ARG, "ssm_scan_fwd_vector_decay: give exactly one of log_decay and A_vec");
    if (work && A_vec != nullptr && dt == nullptr)
        return fail(SSM_ERR_INVALID_ARG, "ssm_scan_fwd_vector_decay: the A_vec form needs dt");
    if (!ssm::recurrent_supported(headdim, dstate, true))
        return fail(SSM_ERR_UNSUPPORTED, "ssm_scan_fwd_vector_decay: dstate must be 4 * 2^k <= 256 and headdim*dstate <= 16384");
    st = check_ptrs(fn, {{"x", x, work, es},
                         {"dt", dt, false, 4},
                         {"log_decay", log_decay, false, 4},
                         {"A_vec", A_vec, false, 4},
                         {"B", Bm, work, es},
                         {"C", Cm, work, es},
                         {"initial_state", initial_state, false, 16},
                         {"final_state", final_state, false, 16},
                         {"seq_idx", seq_idx, false, 4},
                         {"y", y, work, es}});
    if (st != SSM_OK) return st;
    if (!rows) return ok();
    if (!work)  // no tokens: the final state is the initial state (or zero)
        return hip_status(ssm::launch_copy_or_zero_f32(final_state, initial_state,
                                                       batch * nheads * headdim * dstate,
                                                       reinterpret_cast<hipStream_t>(stream)),
                          fn);
    ssm::RecurrentArgs r{};
    r.x = x;
    r.x_sb = seqlen * nheads * headdim;
    r.x_st = nheads * headdim;
    r.x_sc = 1;
    r.dt = dt;
    r.A = nullptr;
    r.Bm = Bm;
    r.B_sb = seqlen * ngroups * dstate;
    r.B_st = ngroups * dstate;
    r.B_sc = 1;
    r.Cm = Cm;
    r.C_sb = r.B_sb;
    r.C_st = r.B_st;
    r.C_sc = 1;
    r.state_in = initial_state;
    r.state_out = final_state;
    r.indices = nullptr;
    r.n_slots = batch;
    r.seq_idx = seq_idx;
    r.y = y;
    r.B = batch;
    r.T = seqlen;
    r.H = nheads;
    r.P = headdim;
    r.G = ngroups;
    r.N = dstate;
    r.log_decay = log_decay;
    r.A_vec = A_vec;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (ssm::vdecay_supported(headdim, dstate))
        return hip_status(ssm::launch_vdecay(r, dtype, s), fn);
    return hip_status(ssm::launch_recurrent(r, dtype, s), fn);
}

namespace {
size_t round256(size_t n) { return (n + 255) / 256 * 256; }
}  // namespace

size_t ssm_conv_scan_fwd_pooled_workspace_size(int64_t batch, int64_t seqlen, int64_t nheads,
                                               int64_t headdim, int64_t ngroups, int64_t dstate,
                                               int64_t width, ssm_dtype_t dtype) {
    if (batch <= 0 || nheads < 1 || headdim < 1 || ngroups < 1 || dstate < 1 || width < 2 ||
        width > 8 || !valid_dtype(dtype))
        return 0;
    const int64_t C_conv = nheads * headdim + 2 * ngroups * dstate;
    const size_t scan = round256(ssm_scan_workspace_size(batch, seqlen, nheads, headdim, ngroups,
                                                         dstate, dtype));
    const size_t hist = round256(static_cast<size_t>(batch * C_conv * (width - 1)) * esize(dtype));
    const size_t st = round256(static_cast<size_t>(batch * nheads * headdim * dstate) * 4);
    return scan + hist + st;
}

ssm_status_t ssm_conv_scan_fwd_pooled(const void* xBC, const float* conv_w,
                                      const float* conv_bias, const float* dt, const float* A,
                                      void* conv_state, float* ssm_state,
                                      const int32_t* state_indices, const int32_t* cache_seqlens,
                                      const int32_t* seq_idx, void* y, int64_t batch,
                                      int64_t seqlen, int64_t nheads, int64_t headdim,
                                      int64_t ngroups, int64_t dstate, int64_t width,
                                      int64_t state_len, int64_t n_slots, ssm_dtype_t dtype,
                                      ssm_act_t act, void* workspace, size_t workspace_bytes,
                                      ssm_stream_t stream) {
    const char* fn = "ssm_conv_scan_fwd_pooled";
    ssm_status_t st = check_scan_dims(fn, batch, seqlen, nheads, headdim, ngroups, dstate, dtype);
    if (st != SSM_OK) return st;
    if (!valid_act(act)) return fail(SSM_ERR_INVALID_ARG, "ssm_conv_scan_fwd_pooled: bad activation");
    if (width < 2 || width > 8)
        return fail(SSM_ERR_UNSUPPORTED, "ssm_conv_scan_fwd_pooled: width must be in [2, 8]");
    if (n_slots < 1 || state_len < width - 1)
        return fail(SSM_ERR_INVALID_ARG,
                    "ssm_conv_scan_fwd_pooled: need n_slots >= 1 and state_len >= width - 1");
    const size_t es = esize(dtype);
    const bool rows = batch > 0;
    // every pointer is checked before the first launch, so a rejected call leaves the pools
    // and the workspace untouched
    st = check_ptrs(fn, {{"xBC", xBC, rows, es},
                         {"conv_w", conv_w, rows, 4},
                         {"conv_bias", conv_bias, false, 4},
                         {"dt", dt, rows, 4},
                         {"A", A, rows, 4},
                         {"conv_state", conv_state, rows, es},
                         {"ssm_state", ssm_state, rows, 4},
                         {"state_indices", state_indices, false, 4},
                         {"cache_seqlens", cache_seqlens, false, 4},
                         {"seq_idx", seq_idx, false, 4},
                         {"y", y, rows, es}});
    if (st != SSM_OK) return st;
    if (!rows) return ok();
    const size_t need = ssm_conv_scan_fwd_pooled_workspace_size(batch, seqlen, nheads, headdim,
                                                                ngroups, dstate, width, dtype);
    if (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 256))
        return fail(SSM_ERR_WORKSPACE, std::string(fn) + ": workspace must be >= " +
                                           std::to_string(need) + " bytes, 256-byte aligned");
    const int64_t C_conv = nheads * headdim + 2 * ngroups * dstate;
    const int64_t per = nheads * headdim * dstate;
    const size_t scan = round256(ssm_scan_workspace_size(batch, seqlen, nheads, headdim, ngroups,
                                                         dstate, dtype));
    const size_t hist_b = round256(static_cast<size_t>(batch * C_conv * (width - 1)) * es);
    uint8_t* base = static_cast<uint8_t*>(workspace);
    void* hist = base + scan;
    float* sstate = reinterpret_cast<float*>(base + scan + hist_b);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    // The chunked scan reads and writes the SSM pool rows itself (no gather or scatter of
    // states); other shapes run the states through the workspace.
    const bool in_pool = ssm::chunked_supported(headdim, dstate, dtype) && aligned(ssm_state, 16);
    const int64_t moved = in_pool ? 0 : per;
    hipError_t e = ssm::launch_pool_gather(conv_state, ssm_state, state_indices, cache_seqlens,
                                           hist, sstate, batch, C_conv, width, state_len, moved,
                                           n_slots, dtype, s);
    if (e != hipSuccess) return hip_status(e, fn);
    if (in_pool)
        st = conv_scan_fwd_impl(fn, xBC, conv_w, conv_bias, hist, nullptr, dt, A, ssm_state,
                                ssm_state, seq_idx, y, batch, seqlen, nheads, headdim, ngroups,
                                dstate, width, dtype, act, scan > 0 ? workspace : nullptr, scan,
                                true, stream, state_indices, n_slots);
    else
        st = ssm_conv_scan_fwd(xBC, conv_w, conv_bias, hist, nullptr, dt, A, sstate, sstate,
                               seq_idx, y, batch, seqlen, nheads, headdim, ngroups, dstate, width,
                               dtype, act, scan > 0 ? workspace : nullptr, scan, stream);
    if (st != SSM_OK) return st;
    return hip_status(ssm::launch_pool_scatter(conv_state, ssm_state, state_indices, cache_seqlens,
                                               xBC, sstate, batch, seqlen, C_conv, state_len,
                                               moved, n_slots, dtype, s),
                      fn);
}

size_t ssm_conv1d_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t channels,
                                     int64_t width) {
    if (batch <= 0 || seqlen <= 0 || channels < 1 || width < 2 || width > 8) return 0;
    return static_cast<size_t>(ssm::conv1d_bwd_workspace_bytes(batch, seqlen, channels, width));
}

ssm_status_t ssm_conv1d_bwd(const void* x, const float* w, const float* bias,
                            const void* initial_state, const int32_t* seq_idx, const void* dout,
                            const void* dfinal_state, void* dx, void* dinitial_state, float* dw,
                            float* dbias, void* workspace, size_t workspace_bytes, int64_t batch,
                            int64_t seqlen, int64_t channels, int64_t width, ssm_dtype_t dtype,
                            ssm_act_t act, ssm_stream_t stream) {
    const char* fn = "ssm_conv1d_bwd";
    if (!valid_dtype(dtype)) return fail(SSM_ERR_INVALID_ARG, "ssm_conv1d_bwd: bad dtype");
    if (!valid_act(act)) return fail(SSM_ERR_INVALID_ARG, "ssm_conv1d_bwd: bad activation");
    if (batch < 0 || seqlen < 0 || channels < 1)
        return fail(SSM_ERR_INVALID_ARG, "ssm_conv1d_bwd: need batch >= 0, seqlen >= 0, channels >= 1");
    if (width < 2 || width > 8)
        return fail(SSM_ERR_UNSUPPORTED, "ssm_conv1d_bwd: width must be in [2, 8]");
    const size_t es = esize(dtype);
    const bool rows = batch > 0;
    const bool work = rows && seqlen > 0;
    ssm_status_t st = check_ptrs(fn, {{"x", x, work, es},
                                      {"w", w, work, 4},
                                      {"bias", bias, false, 4},
                                      {"initial_state", initial_state, false, es},
                                      {"seq_idx", seq_idx, false, 4},
                                      {"dout", dout, work, es},
                                      {"dfinal_state", dfinal_state, false, es},
                                      {"dx", dx, work, es},
                                      {"dinitial_state", dinitial_state, false, es},
                                      {"dw", dw, rows, 4},
                                      {"dbias", dbias, false, 4},
                                      {"workspace", workspace, false, 4}});
    if (st != SSM_OK) return st;
    if (!rows) return ok();
    const size_t need = ssm_conv1d_bwd_workspace_size(batch, seqlen, channels, width);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need))
        return fail(SSM_ERR_WORKSPACE, "ssm_conv1d_bwd: workspace missing or smaller than "
                                       "ssm_conv1d_bwd_workspace_size");
    return hip_status(ssm::launch_conv1d_bwd(x, w, bias, initial_state, seq_idx, dout, dfinal_state,
                                             dx, dinitial_state, dw, dbias, workspace, batch, seqlen,
                                             channels, width, dtype, act,
                                             reinterpret_cast<hipStream_t>(stream)),
                      fn);
}

ssm_status_t ssm_scan_bwd_initial_state(const float* dt, const float* A, const void* C,
                                        const void* dy, const int32_t* seq_idx,
                                        const float* dfinal_state, float* dinitial_state,
                                        int64_t batch, int64_t seqlen, int64_t nheads,
                                        int64_t headdim, int64_t ngroups, int64_t dstate,
                                        ssm_dtype_t dtype, ssm_stream_t stream) {
    const char* fn = "ssm_scan_bwd_initial_state";
    ssm_status_t st = check_scan_dims(fn, batch, seqlen, nheads, headdim, ngroups, dstate, dtype);
    if (st != SSM_OK) return st;
    const size_t es = esize(dtype);
    const bool rows = batch > 0;
    const bool work = rows && seqlen > 0;
    st = check_ptrs(fn, {{"dt", dt, work, 4},
                         {"A", A, rows, 4},
                         {"C", C, work, es},
                         {"dy", dy, work, es},
                         {"seq_idx", seq_idx, false, 4},
                         {"dfinal_state", dfinal_state, false, 4},
                         {"dinitial_state", dinitial_state, rows, 4}});
    if (st != SSM_OK) return st;
    if (!rows) return ok();
    return hip_status(ssm::launch_scan_bwd_h0(dt, A, C, seq_idx, dy, dfinal_state, dinitial_state,
                                              batch, seqlen, nheads, headdim, ngroups, dstate,
                                              dtype, reinterpret_cast<hipStream_t>(stream)),
                      fn);
}

namespace {

ssm_status_t check_norm_dims(const char* fn, int64_t rows, int64_t channels, int64_t ngroups,
                             float eps, int32_t kind, int dtype) {
    if (!valid_dtype(dtype)) return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": bad dtype");
    if (kind != SSM_NORM_RMS && kind != SSM_NORM_LAYER)
        return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": bad norm kind");
    if (rows < 0 || channels < 1 || ngroups < 1 || channels % ngroups != 0)
        return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": need rows >= 0 and channels a positive multiple of ngroups");
    if (!(eps >= 0.0f)) return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": eps must be >= 0");
    if (channels / ngroups > 16384)
        return fail(SSM_ERR_UNSUPPORTED, std::string(fn) + ": channels / ngroups must be <= 16384");
    if (ngroups > 0x7FFFFFFF || channels > (int64_t{1} << 36))
        return fail(SSM_ERR_UNSUPPORTED, std::string(fn) + ": too many channels");
    return SSM_OK;
}
ssm_status_t check_row(const char* fn, const char* name, const void* p, int64_t row, int64_t rows,
                       int64_t least) {
    if (p == nullptr || rows <= 1 || row >= least) return SSM_OK;
    return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": " + name + " row stride below " + std::to_string(least));
}

}  // namespace

ssm_status_t ssm_norm_fwd(const void* x, int64_t x_row, const void* z, int64_t z_row,
                          const float* weight, const float* bias, void* out, int64_t out_row,
                          int64_t rows, int64_t channels, int64_t ngroups, float eps,
                          ssm_norm_t kind, int32_t norm_before_gate, ssm_dtype_t dtype,
                          ssm_stream_t stream) {
    const char* fn = "ssm_norm_fwd";
    ssm_status_t st = check_norm_dims(fn, rows, channels, ngroups, eps, kind, dtype);
    if (st != SSM_OK) return st;
    const size_t es = esize(dtype);
    const bool work = rows > 0;
    st = check_ptrs(fn, {{"x", x, work, es},
                         {"z", z, false, es},
                         {"weight", weight, false, 4},
                         {"bias", bias, false, 4},
                         {"out", out, work, es}});
    if (st == SSM_OK) st = check_row(fn, "x", x, x_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "z", z, z_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "out", out, out_row, rows, channels);
    if (st != SSM_OK) return st;
    if (!work) return ok();
    ssm::NormCall c{};
    c.x = x;
    c.x_row = x_row;
    c.z = z;
    c.z_row = z_row;
    c.w = weight;
    c.b = bias;
    c.out = out;
    c.out_row = out_row;
    c.rows = rows;
    c.channels = channels;
    c.groups = ngroups;
    c.eps = eps;
    c.layer = kind == SSM_NORM_LAYER;
    c.gate_after = norm_before_gate != 0;
    c.dtype = dtype;
    return hip_status(ssm::launch_norm_fwd(c, reinterpret_cast<hipStream_t>(stream)), fn);
}

size_t ssm_norm_bwd_workspace_size(int64_t rows, int64_t channels, int64_t ngroups) {
    if (rows <= 0 || channels < 1 || ngroups < 1 || channels % ngroups != 0 || channels > (int64_t{1} << 36)) return 0;
    return static_cast<size_t>(2 * ssm::norm_partial_rows(rows, channels, ngroups) * channels) * 4;
}

ssm_status_t ssm_norm_bwd(const void* x, int64_t x_row, const void* z, int64_t z_row,
                          const void* dout, int64_t dout_row, const float* weight,
                          const float* bias, void* dx, int64_t dx_row, void* dz, int64_t dz_row,
                          float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                          int64_t rows, int64_t channels, int64_t ngroups, float eps,
                          ssm_norm_t kind, int32_t norm_before_gate, ssm_dtype_t dtype,
                          ssm_stream_t stream) {
    const char* fn = "ssm_norm_bwd";
    ssm_status_t st = check_norm_dims(fn, rows, channels, ngroups, eps, kind, dtype);
    if (st != SSM_OK) return st;
    const size_t es = esize(dtype);
    const bool work = rows > 0;
    if (z == nullptr) dz = nullptr;
    st = check_ptrs(fn, {{"x", x, work, es},
                         {"z", z, false, es},
                         {"dout", dout, work, es},
                         {"weight", weight, false, 4},
                         {"bias", bias, false, 4},
                         {"dx", dx, work, es},
                         {"dz", dz, false, es},
                         {"dweight", dweight, false, 4},
                         {"dbias", dbias, false, 4},
                         {"workspace", workspace, false, 4}});
    if (st == SSM_OK) st = check_row(fn, "x", x, x_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "z", z, z_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "dout", dout, dout_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "dx", dx, dx_row, rows, channels);
    if (st == SSM_OK) st = check_row(fn, "dz", dz, dz_row, rows, channels);
    if (st != SSM_OK) return st;
    if (work && (dweight || dbias)) {
        const size_t need = ssm_norm_bwd_workspace_size(rows, channels, ngroups);
        if (workspace == nullptr || workspace_bytes < need)
            return fail(SSM_ERR_WORKSPACE, "ssm_norm_bwd: workspace missing or smaller than "
                                           "ssm_norm_bwd_workspace_size");
    }
    if (!work && !dweight && !dbias) return ok();
    ssm::NormCall c{};
    c.x = x;
    c.x_row = x_row;
    c.z = z;
    c.z_row = z_row;
    c.dout = dout;
    c.dout_row = dout_row;
    c.w = weight;
    c.b = bias;
    c.dx = dx;
    c.dx_row = dx_row;
    c.dz = dz;
    c.dz_row = dz_row;
    c.dw = dweight;
    c.db = dbias;
    c.workspace = workspace;
    c.rows = rows;
    c.channels = channels;
    c.groups = ngroups;
    c.eps = eps;
    c.layer = kind == SSM_NORM_LAYER;
    c.gate_after = norm_before_gate != 0;
    c.dtype = dtype;
    return hip_status(ssm::launch_norm_bwd(c, reinterpret_cast<hipStream_t>(stream)), fn);
}

// sizes whose products do not leave 63 bits
static bool scan_bwd_sizes_fit(int64_t batch, int64_t seqlen, int64_t nheads) {
    const int64_t most = int64_t{1} << 31;
    return batch < most && seqlen < most && nheads < most &&
           (batch == 0 || seqlen == 0 || nheads <= (most << 20) / batch / seqlen);
}

size_t ssm_scan_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                                   int64_t ngroups, int64_t dstate, ssm_dtype_t dtype) {
    if (batch <= 0 || seqlen <= 0 || nheads < 1 || headdim < 1 || ngroups < 1 || dstate < 1 ||
        nheads % ngroups != 0 || !valid_dtype(dtype) || !ssm::recurrent_supported(headdim, dstate) ||
        !scan_bwd_sizes_fit(batch, seqlen, nheads))
        return 0;
    return ssm::scan_bwd_workspace_bytes(batch, seqlen, nheads, headdim, ngroups, dstate, dtype);
}

ssm_status_t ssm_scan_bwd(const void* x, const float* dt, const float* A, const void* Bm,
                          const void* Cm, const void* dy, const float* initial_state,
                          const float* dfinal_state, const int32_t* seq_idx, void* dx, float* ddt,
                          float* dA, void* dB, void* dC, float* dinitial_state, int64_t batch,
                          int64_t seqlen, int64_t nheads, int64_t headdim, int64_t ngroups,
                          int64_t dstate, ssm_dtype_t dtype, void* workspace,
                          size_t workspace_bytes, ssm_stream_t stream) {
    const char* fn = "ssm_scan_bwd";
    ssm_status_t st = check_scan_dims(fn, batch, seqlen, nheads, headdim, ngroups, dstate, dtype);
    if (st != SSM_OK) return st;
    if (!ssm::recurrent_supported(headdim, dstate))
        return fail(SSM_ERR_UNSUPPORTED, "ssm_scan_bwd: headdim and dstate must be sizes that ssm_scan_fwd takes (dstate 4 * 2^k <= 256, headdim*dstate <= 32768)");
    if (!scan_bwd_sizes_fit(batch, seqlen, nheads))
        return fail(SSM_ERR_UNSUPPORTED, "ssm_scan_bwd: batch, seqlen or nheads too large");
    const size_t es = esize(dtype);
    const bool work = batch > 0 && seqlen > 0;
    st = check_ptrs(fn, {{"x", x, work, es},
                         {"dt", dt, work, 4},
                         {"A", A, work, 4},
                         {"Bm", Bm, work, es},
                         {"Cm", Cm, work, es},
                         {"dy", dy, work, es},
                         {"initial_state", initial_state, false, 16},
                         {"dfinal_state", dfinal_state, false, 16},
                         {"seq_idx", seq_idx, false, 4},
                         {"dx", dx, work, es},
                         {"ddt", ddt, work, 4},
                         {"dA", dA, true, 4},
                         {"dB", dB, work, es},
                         {"dC", dC, work, es},
                         {"dinitial_state", dinitial_state, false, 16}});
    if (st != SSM_OK) return st;
    if (dinitial_state != nullptr && dinitial_state == dfinal_state)
        return fail(SSM_ERR_INVALID_ARG, "ssm_scan_bwd: dinitial_state must not be dfinal_state");
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (!work)
        return hip_status(ssm::launch_scan_bwd_empty(dfinal_state, dinitial_state, dA,
                                                     batch * nheads * headdim * dstate, nheads, s),
                          fn);
    if (ssm::scan_bwd_blocks(batch, seqlen, nheads, headdim, ngroups, dstate) > 0x7FFFFFFF)
        return fail(SSM_ERR_UNSUPPORTED, "ssm_scan_bwd: tensors too large for one call");
    const size_t need = ssm_scan_bwd_workspace_size(batch, seqlen, nheads, headdim, ngroups, dstate, dtype);
    if (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 256))
        return fail(SSM_ERR_WORKSPACE, "ssm_scan_bwd: workspace must be >= " + std::to_string(need) +
                                           " bytes, 256-byte aligned");
    ssm::ScanBwdArgs a{};
    a.x = x;
    a.dt = dt;
    a.A = A;
    a.Bm = Bm;
    a.C = Cm;
    a.dy = dy;
    a.h0 = initial_state;
    a.dhT = dfinal_state;
    a.seq = seq_idx;
    a.dx = dx;
    a.ddt = ddt;
    a.dA = dA;
    a.dB = dB;
    a.dC = dC;
    a.dh0 = dinitial_state;
    a.x_row = a.dy_row = a.dx_row = nheads * headdim;
    a.b_row = a.c_row = a.db_row = a.dc_row = ngroups * dstate;
    a.B = batch;
    a.L = seqlen;
    a.H = nheads;
    a.P = headdim;
    a.G = ngroups;
    a.N = dstate;
    return hip_status(ssm::launch_scan_bwd(a, workspace, dtype, s), fn);
}

namespace {

// sizes whose products below do not leave 63 bits, nor their grid 31
bool gscan_sizes_fit(int64_t batch, int64_t seqlen, int64_t channels) {
    const int64_t most = int64_t{1} << 31;
    return batch < most && seqlen < most && channels < most && (batch == 0 || (channels + 63) / 64 <= most / batch);
}

ssm_status_t check_gscan_dims(const char* fn, int64_t batch, int64_t seqlen, int64_t channels,
                              int32_t form, int dtype) {
    if (!valid_dtype(dtype)) return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": bad dtype");
    if (form != SSM_GATE_LOG && form != SSM_GATE_SIGMOID)
        return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": bad gate form");
    if (batch < 0 || seqlen < 0 || channels < 1)
        return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": need batch >= 0, tokens >= 0, channels >= 1");
    if (!gscan_sizes_fit(batch, seqlen, channels))
        return fail(SSM_ERR_UNSUPPORTED, std::string(fn) + ": batch, tokens or channels too large");
    return SSM_OK;
}

}  // namespace

size_t ssm_gated_scan_fwd_workspace_size(int64_t batch, int64_t seqlen, int64_t channels) {
    if (batch <= 0 || seqlen <= 0 || channels < 1 || !gscan_sizes_fit(batch, seqlen, channels)) return 0;
    return ssm::gscan_workspace_bytes(batch, seqlen, channels, false);
}

size_t ssm_gated_scan_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t channels) {
    if (batch <= 0 || seqlen <= 0 || channels < 1 || !gscan_sizes_fit(batch, seqlen, channels)) return 0;
    return ssm::gscan_workspace_bytes(batch, seqlen, channels, true);
}

ssm_status_t ssm_gated_scan_fwd(const void* x, int64_t x_row, const void* gate, int64_t gate_row,
                                const float* initial_state, float* final_state,
                                const int32_t* seq_idx, void* y, int64_t y_row, int64_t batch,
                                int64_t seqlen, int64_t channels, ssm_gate_t form,
                                ssm_dtype_t dtype, void* workspace, size_t workspace_bytes,
                                ssm_stream_t stream) {
    const char* fn = "ssm_gated_scan_fwd";
    ssm_status_t st = check_gscan_dims(fn, batch, seqlen, channels, form, dtype);
    if (st != SSM_OK) return st;
    const size_t es = esize(dtype);
    const bool work = batch > 0 && seqlen > 0;
    const int64_t rows = batch * seqlen;
    st = check_ptrs(fn, {{"x", x, work, es},
                         {"gate", gate, work, es},
                         {"initial_state", initial_state, false, 4},
                         {"final_state", final_state, false, 4},
                         {"seq_idx", seq_idx, false, 4},
                         {"y", y, work, es},
                         {"workspace", workspace, false, 4}});
    if (st == SSM_OK) st = check_row(fn, "x", x, x_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "gate", gate, gate_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "y", y, y_row, rows, channels);
    if (st != SSM_OK) return st;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (batch == 0) return ok();
    if (seqlen == 0)
        return hip_status(ssm::launch_copy_or_zero_f32(final_state, initial_state, batch * channels, s), fn);
    if (ssm::gscan_blocks(batch, seqlen, channels) > 0x7FFFFFFF)
        return fail(SSM_ERR_UNSUPPORTED, std::string(fn) + ": too many rows and channels");
    const size_t need = ssm_gated_scan_fwd_workspace_size(batch, seqlen, channels);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need))
        return fail(SSM_ERR_WORKSPACE, std::string(fn) + ": workspace missing or smaller than "
                                       "ssm_gated_scan_fwd_workspace_size");
    ssm::GscanCall c{};
    c.x = x;
    c.x_row = x_row;
    c.gate = gate;
    c.gate_row = gate_row;
    c.y = y;
    c.y_row = y_row;
    c.h0 = initial_state;
    c.final_state = final_state;
    c.seq = seq_idx;
    c.workspace = workspace;
    c.B = batch;
    c.L = seqlen;
    c.C = channels;
    c.sigmoid = form == SSM_GATE_SIGMOID;
    c.dtype = dtype;
    return hip_status(ssm::launch_gscan_fwd(c, s), fn);
}

ssm_status_t ssm_gated_scan_bwd(const void* x, int64_t x_row, const void* gate, int64_t gate_row,
                                const void* dy, int64_t dy_row, const float* initial_state,
                                const float* dfinal_state, const int32_t* seq_idx, void* dx,
                                int64_t dx_row, void* dgate, int64_t dgate_row,
                                float* dinitial_state, int64_t batch, int64_t seqlen,
                                int64_t channels, ssm_gate_t form, ssm_dtype_t dtype,
                                void* workspace, size_t workspace_bytes, ssm_stream_t stream) {
    const char* fn = "ssm_gated_scan_bwd";
    ssm_status_t st = check_gscan_dims(fn, batch, seqlen, channels, form, dtype);
    if (st != SSM_OK) return st;
    const size_t es = esize(dtype);
    const bool work = batch > 0 && seqlen > 0;
    const int64_t rows = batch * seqlen;
    st = check_ptrs(fn, {{"x", x, work, es},
                         {"gate", gate, work, es},
                         {"dy", dy, work, es},
                         {"initial_state", initial_state, false, 4},
                         {"dfinal_state", dfinal_state, false, 4},
                         {"seq_idx", seq_idx, false, 4},
                         {"dx", dx, work, es},
                         {"dgate", dgate, work, es},
                         {"dinitial_state", dinitial_state, false, 4},
                         {"workspace", workspace, false, 4}});
    if (st == SSM_OK) st = check_row(fn, "x", x, x_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "gate", gate, gate_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "dy", dy, dy_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "dx", dx, dx_row, rows, channels);
    if (st == SSM_OK) st = check_row(fn, "dgate", dgate, dgate_row, rows, channels);
    if (st != SSM_OK) return st;
    if (dinitial_state != nullptr && dinitial_state == dfinal_state)
        return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": dinitial_state must not be dfinal_state");
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (batch == 0) return ok();
    if (seqlen == 0)
        return hip_status(ssm::launch_copy_or_zero_f32(dinitial_state, dfinal_state, batch * channels, s), fn);
    if (ssm::gscan_blocks(batch, seqlen, channels) > 0x7FFFFFFF)
        return fail(SSM_ERR_UNSUPPORTED, std::string(fn) + ": too many rows and channels");
    const size_t need = ssm_gated_scan_bwd_workspace_size(batch, seqlen, channels);
    if (workspace == nullptr || workspace_bytes < need)
        return fail(SSM_ERR_WORKSPACE, std::string(fn) + ": workspace missing or smaller than "
                                       "ssm_gated_scan_bwd_workspace_size");
    ssm::GscanCall c{};
    c.x = x;
    c.x_row = x_row;
    c.gate = gate;
    c.gate_row = gate_row;
    c.dy = dy;
    c.dy_row = dy_row;
    c.dx = dx;
    c.dx_row = dx_row;
    c.dgate = dgate;
    c.dgate_row = dgate_row;
    c.h0 = initial_state;
    c.dhT = dfinal_state;
    c.dh0 = dinitial_state;
    c.seq = seq_idx;
    c.workspace = workspace;
    c.B = batch;
    c.L = seqlen;
    c.C = channels;
    c.sigmoid = form == SSM_GATE_SIGMOID;
    c.dtype = dtype;
    return hip_status(ssm::launch_gscan_bwd(c, s), fn);
}

ssm_status_t ssm_gated_scan_step(const void* x, int64_t x_row, const void* gate, int64_t gate_row,
                                 float* state, const int32_t* state_indices, void* y,
                                 int64_t y_row, int64_t batch, int64_t n_new, int64_t channels,
                                 int64_t n_slots, ssm_gate_t form, ssm_dtype_t dtype,
                                 ssm_stream_t stream) {
    const char* fn = "ssm_gated_scan_step";
    ssm_status_t st = check_gscan_dims(fn, batch, n_new, channels, form, dtype);
    if (st != SSM_OK) return st;
    if (n_slots < 1) return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": n_slots must be >= 1");
    const size_t es = esize(dtype);
    const bool work = batch > 0 && n_new > 0;
    const int64_t rows = batch * n_new;
    st = check_ptrs(fn, {{"x", x, work, es},
                         {"gate", gate, work, es},
                         {"state", state, work, 4},
                         {"state_indices", state_indices, false, 4},
                         {"y", y, work, es}});
    if (st == SSM_OK) st = check_row(fn, "x", x, x_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "gate", gate, gate_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "y", y, y_row, rows, channels);
    if (st != SSM_OK) return st;
    if (!work) return ok();
    if ((batch * channels + 255) / 256 > 0x7FFFFFFF)
        return fail(SSM_ERR_UNSUPPORTED, std::string(fn) + ": too many rows and channels");
    ssm::GscanCall c{};
    c.x = x;
    c.x_row = x_row;
    c.gate = gate;
    c.gate_row = gate_row;
    c.y = y;
    c.y_row = y_row;
    c.B = batch;
    c.L = n_new;
    c.C = channels;
    c.sigmoid = form == SSM_GATE_SIGMOID;
    c.dtype = dtype;
    return hip_status(ssm::launch_gscan_step(c, state, state_indices, n_slots,
                                             reinterpret_cast<hipStream_t>(stream)),
                      fn);
}

namespace {

// what the three calls of the gated delta rule share: sizes, then the token rows' strides
ssm_status_t check_delta_dims(const char* fn, int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                              int64_t ngroups, int64_t dstate, float scale, int dtype) {
    ssm_status_t st = check_scan_dims(fn, batch, seqlen, nheads, headdim, ngroups, dstate, dtype);
    if (st != SSM_OK) return st;
    if (dstate % 4 != 0 || dstate > 256)
        return fail(SSM_ERR_UNSUPPORTED, std::string(fn) + ": dstate must be a multiple of 4, at most 256");
    if (headdim > 65536) return fail(SSM_ERR_UNSUPPORTED, std::string(fn) + ": headdim must be at most 65536");
    if (!std::isfinite(scale)) return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": scale must be finite");
    return SSM_OK;
}
// sizes whose products below do not leave 63 bits, nor their numbers of blocks 31
bool delta_sizes_fit(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim) {
    const int64_t most = int64_t{1} << 31;
    if (batch >= most || seqlen >= most || nheads >= most) return false;
    if (batch == 0) return true;
    return nheads < most / batch && (seqlen + 31) / 32 < most / (batch * nheads) &&
           (headdim + 15) / 16 < most / (batch * nheads);
}
// the same for the calls over long rows, and grids that can be launched
bool delta_rows_fit(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim, int64_t ngroups, int64_t dstate,
                    ssm_dtype_t dtype, bool bwd) {
    return delta_sizes_fit(batch, seqlen, nheads, headdim) &&
           (batch == 0 || seqlen == 0 || ssm::delta_launches_fit(batch, seqlen, nheads, headdim, ngroups, dstate, dtype, bwd));
}

}  // namespace

size_t ssm_delta_scan_fwd_workspace_size(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                                         int64_t ngroups, int64_t dstate, ssm_dtype_t dtype) {
    if (batch <= 0 || seqlen <= 0 ||
        check_delta_dims("ssm_delta_scan_fwd_workspace_size", batch, seqlen, nheads, headdim, ngroups, dstate, 1.0f, dtype) != SSM_OK ||
        !delta_rows_fit(batch, seqlen, nheads, headdim, ngroups, dstate, dtype, false))
        return 0;
    return ssm::delta_fwd_workspace_bytes(batch, seqlen, nheads, headdim, ngroups, dstate, dtype);
}

size_t ssm_delta_scan_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                                         int64_t ngroups, int64_t dstate, ssm_dtype_t dtype) {
    if (batch <= 0 || seqlen <= 0 ||
        check_delta_dims("ssm_delta_scan_bwd_workspace_size", batch, seqlen, nheads, headdim, ngroups, dstate, 1.0f, dtype) != SSM_OK ||
        !delta_rows_fit(batch, seqlen, nheads, headdim, ngroups, dstate, dtype, true))
        return 0;
    return ssm::delta_bwd_workspace_bytes(batch, seqlen, nheads, headdim, ngroups, dstate, dtype);
}

ssm_status_t ssm_delta_scan_fwd(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
                                int64_t v_row, const float* beta, const float* gate, float scale,
                                const float* initial_state, float* final_state, const int32_t* seq_idx,
                                void* y, int64_t y_row, int64_t batch, int64_t seqlen, int64_t nheads,
                                int64_t headdim, int64_t ngroups, int64_t dstate, ssm_dtype_t dtype,
                                void* workspace, size_t workspace_bytes, ssm_stream_t stream) {
    const char* fn = "ssm_delta_scan_fwd";
    ssm_status_t st = check_delta_dims(fn, batch, seqlen, nheads, headdim, ngroups, dstate, scale, dtype);
    if (st != SSM_OK) return st;
    if (!delta_rows_fit(batch, seqlen, nheads, headdim, ngroups, dstate, dtype, false))
        return fail(SSM_ERR_UNSUPPORTED, std::string(fn) + ": batch, seqlen, nheads or headdim too large");
    const size_t es = esize(dtype);
    const bool work = batch > 0 && seqlen > 0;
    const int64_t rows = batch * seqlen;
    st = check_ptrs(fn, {{"q", q, work, es},
                         {"k", k, work, es},
                         {"v", v, work, es},
                         {"beta", beta, work, 4},
                         {"gate", gate, false, 4},
                         {"initial_state", initial_state, false, 16},
                         {"final_state", final_state, false, 16},
                         {"seq_idx", seq_idx, false, 4},
                         {"y", y, work, es}});
    if (st == SSM_OK) st = check_row(fn, "q", q, q_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "k", k, k_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "v", v, v_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "y", y, y_row, rows, nheads * headdim);
    if (st != SSM_OK) return st;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (!work)
        return hip_status(ssm::launch_copy_or_zero_f32(final_state, initial_state, batch * nheads * headdim * dstate, s), fn);
    const size_t need = ssm_delta_scan_fwd_workspace_size(batch, seqlen, nheads, headdim, ngroups, dstate, dtype);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 256)))
        return fail(SSM_ERR_WORKSPACE, std::string(fn) + ": workspace must be >= " + std::to_string(need) +
                                           " bytes, 256-byte aligned");
    ssm::DeltaArgs a{};
    a.q = q;
    a.q_row = q_row;
    a.k = k;
    a.k_row = k_row;
    a.v = v;
    a.v_row = v_row;
    a.beta = beta;
    a.gate = gate;
    a.scale = scale;
    a.h0 = initial_state;
    a.final_state = final_state;
    a.seq = seq_idx;
    a.y = y;
    a.y_row = y_row;
    a.B = batch;
    a.L = seqlen;
    a.H = nheads;
    a.P = headdim;
    a.G = ngroups;
    a.N = dstate;
    return hip_status(ssm::launch_delta_fwd(a, workspace, dtype, s), fn);
}

ssm_status_t ssm_delta_scan_bwd(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
                                int64_t v_row, const float* beta, const float* gate, float scale,
                                const void* dy, int64_t dy_row, const float* initial_state,
                                const float* dfinal_state, const int32_t* seq_idx, void* dq, int64_t dq_row,
                                void* dk, int64_t dk_row, void* dv, int64_t dv_row, float* dbeta,
                                float* dgate, float* dinitial_state, int64_t batch, int64_t seqlen,
                                int64_t nheads, int64_t headdim, int64_t ngroups, int64_t dstate,
                                ssm_dtype_t dtype, void* workspace, size_t workspace_bytes,
                                ssm_stream_t stream) {
    const char* fn = "ssm_delta_scan_bwd";
    ssm_status_t st = check_delta_dims(fn, batch, seqlen, nheads, headdim, ngroups, dstate, scale, dtype);
    if (st != SSM_OK) return st;
    if (!delta_rows_fit(batch, seqlen, nheads, headdim, ngroups, dstate, dtype, true))
        return fail(SSM_ERR_UNSUPPORTED, std::string(fn) + ": batch, seqlen, nheads or headdim too large");
    const size_t es = esize(dtype);
    const bool work = batch > 0 && seqlen > 0;
    const int64_t rows = batch * seqlen;
    st = check_ptrs(fn, {{"q", q, work, es},
                         {"k", k, work, es},
                         {"v", v, work, es},
                         {"beta", beta, work, 4},
                         {"gate", gate, false, 4},
                         {"dy", dy, work, es},
                         {"initial_state", initial_state, false, 16},
                         {"dfinal_state", dfinal_state, false, 16},
                         {"seq_idx", seq_idx, false, 4},
                         {"dq", dq, work, es},
                         {"dk", dk, work, es},
                         {"dv", dv, work, es},
                         {"dbeta", dbeta, work, 4},
                         {"dgate", dgate, false, 4},
                         {"dinitial_state", dinitial_state, false, 16}});
    if (st == SSM_OK) st = check_row(fn, "q", q, q_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "k", k, k_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "v", v, v_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "dy", dy, dy_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "dq", dq, dq_row, rows, ngroups * dstate);
    if (st == SSM_OK) st = check_row(fn, "dk", dk, dk_row, rows, ngroups * dstate);
    if (st == SSM_OK) st = check_row(fn, "dv", dv, dv_row, rows, nheads * headdim);
    if (st != SSM_OK) return st;
    if (dinitial_state != nullptr && dinitial_state == dfinal_state)
        return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": dinitial_state must not be dfinal_state");
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (!work)
        return hip_status(ssm::launch_copy_or_zero_f32(dinitial_state, dfinal_state, batch * nheads * headdim * dstate, s), fn);
    const size_t need = ssm_delta_scan_bwd_workspace_size(batch, seqlen, nheads, headdim, ngroups, dstate, dtype);
    if (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 256))
        return fail(SSM_ERR_WORKSPACE, std::string(fn) + ": workspace must be >= " + std::to_string(need) +
                                           " bytes, 256-byte aligned");
    ssm::DeltaArgs a{};
    a.q = q;
    a.q_row = q_row;
    a.k = k;
    a.k_row = k_row;
    a.v = v;
    a.v_row = v_row;
    a.beta = beta;
    a.gate = gate;
    a.scale = scale;
    a.dy = dy;
    a.dy_row = dy_row;
    a.h0 = initial_state;
    a.dhT = dfinal_state;
    a.seq = seq_idx;
    a.dq = dq;
    a.dq_row = dq_row;
    a.dk = dk;
    a.dk_row = dk_row;
    a.dv = dv;
    a.dv_row = dv_row;
    a.dbeta = dbeta;
    a.dgate = dgate;
    a.dh0 = dinitial_state;
    a.B = batch;
    a.L = seqlen;
    a.H = nheads;
    a.P = headdim;
    a.G = ngroups;
    a.N = dstate;
    return hip_status(ssm::launch_delta_bwd(a, workspace, dtype, s), fn);
}

ssm_status_t ssm_delta_scan_step(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
                                 int64_t v_row, const float* beta, const float* gate, float scale,
                                 float* state, const int32_t* state_indices, void* y, int64_t y_row,
                                 int64_t batch, int64_t n_new, int64_t nheads, int64_t headdim,
                                 int64_t ngroups, int64_t dstate, int64_t n_slots, ssm_dtype_t dtype,
                                 ssm_stream_t stream) {
    const char* fn = "ssm_delta_scan_step";
    ssm_status_t st = check_delta_dims(fn, batch, n_new, nheads, headdim, ngroups, dstate, scale, dtype);
    if (st != SSM_OK) return st;
    if (n_slots < 1) return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": n_slots must be >= 1");
    if (!delta_sizes_fit(batch, n_new, nheads, headdim))
        return fail(SSM_ERR_UNSUPPORTED, std::string(fn) + ": batch, n_new, nheads or headdim too large");
    const size_t es = esize(dtype);
    const bool work = batch > 0 && n_new > 0;
    const int64_t rows = batch * n_new;
    st = check_ptrs(fn, {{"q", q, work, es},
                         {"k", k, work, es},
                         {"v", v, work, es},
                         {"beta", beta, work, 4},
                         {"gate", gate, false, 4},
                         {"state", state, work, 16},
                         {"state_indices", state_indices, false, 4},
                         {"y", y, work, es}});
    if (st == SSM_OK) st = check_row(fn, "q", q, q_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "k", k, k_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "v", v, v_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "y", y, y_row, rows, nheads * headdim);
    if (st != SSM_OK) return st;
    if (!work) return ok();
    ssm::DeltaStep d{};
    d.a.q = q;
    d.a.q_row = q_row;
    d.a.k = k;
    d.a.k_row = k_row;
    d.a.v = v;
    d.a.v_row = v_row;
    d.a.beta = beta;
    d.a.gate = gate;
    d.a.scale = scale;
    d.a.y = y;
    d.a.y_row = y_row;
    d.a.B = batch;
    d.a.L = n_new;
    d.a.H = nheads;
    d.a.P = headdim;
    d.a.G = ngroups;
    d.a.N = dstate;
    d.state = state;
    d.slots = state_indices;
    d.n_slots = n_slots;
    return hip_status(ssm::launch_delta_step(d, dtype, reinterpret_cast<hipStream_t>(stream)), fn);
}

namespace {

ssm_status_t check_qk_norm_dims(const char* fn, int64_t batch, int64_t seqlen, int64_t nheads_q, int64_t nheads_k,
                                int64_t headdim, int64_t rotary_dim, const float* inv_freq, float eps,
                                int32_t kind, int dtype) {
    if (!valid_dtype(dtype)) return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": bad dtype");
    if (kind != SSM_QK_NORM_L2 && kind != SSM_QK_NORM_RMS)
        return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": bad norm kind");
    if (batch < 0 || seqlen < 0 || nheads_q < 1 || nheads_k < 1 || headdim < 1)
        return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": need batch >= 0, seqlen >= 0, heads and headdim >= 1");
    if (rotary_dim < 0 || rotary_dim % 2 != 0 || rotary_dim > headdim)
        return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": rotary_dim must be even and at most headdim");
    if (rotary_dim > 0 && inv_freq == nullptr)
        return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": inv_freq is NULL");
    if (!(eps >= 0.0f)) return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": eps must be >= 0");
    if (headdim > 256) return fail(SSM_ERR_UNSUPPORTED, std::string(fn) + ": headdim must be at most 256");
    const int64_t most = int64_t{1} << 31;
    if (batch >= most || seqlen >= most || (batch > 0 && seqlen >= most / batch) || nheads_q >= most / 256 || nheads_k >= most / 256)
        return fail(SSM_ERR_UNSUPPORTED, std::string(fn) + ": too many tokens or heads");
    return SSM_OK;
}

}  // namespace

ssm_status_t ssm_qk_norm_fwd(const void* q, int64_t q_row, const void* k, int64_t k_row, const float* q_weight,
                             const float* k_weight, const float* inv_freq, const int32_t* positions,
                             void* q_out, int64_t q_out_row, void* k_out, int64_t k_out_row, int64_t batch,
                             int64_t seqlen, int64_t nheads_q, int64_t nheads_k, int64_t headdim,
                             int64_t rotary_dim, int32_t interleaved, float eps, ssm_qk_norm_t kind,
                             ssm_dtype_t dtype, ssm_stream_t stream) {
    const char* fn = "ssm_qk_norm_fwd";
    ssm_status_t st = check_qk_norm_dims(fn, batch, seqlen, nheads_q, nheads_k, headdim, rotary_dim, inv_freq, eps, kind, dtype);
    if (st != SSM_OK) return st;
    const size_t es = esize(dtype);
    const int64_t rows = batch * seqlen;
    const bool work = rows > 0;
    st = check_ptrs(fn, {{"q", q, work, es},
                         {"k", k, work, es},
                         {"q_weight", q_weight, false, 4},
                         {"k_weight", k_weight, false, 4},
                         {"inv_freq", inv_freq, false, 4},
                         {"positions", positions, false, 4},
                         {"q_out", q_out, work, es},
                         {"k_out", k_out, work, es}});
    if (st == SSM_OK) st = check_row(fn, "q", q, q_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "k", k, k_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "q_out", q_out, q_out_row, rows, nheads_q * headdim);
    if (st == SSM_OK) st = check_row(fn, "k_out", k_out, k_out_row, rows, nheads_k * headdim);
    if (st != SSM_OK) return st;
    if (!work) return ok();
    ssm::QkNormCall c{};
    c.x[0] = q;
    c.x[1] = k;
    c.x_row[0] = q_row;
    c.x_row[1] = k_row;
    c.out[0] = q_out;
    c.out[1] = k_out;
    c.out_row[0] = q_out_row;
    c.out_row[1] = k_out_row;
    c.w[0] = q_weight;
    c.w[1] = k_weight;
    c.heads[0] = nheads_q;
    c.heads[1] = nheads_k;
    c.tokens = rows;
    c.L = seqlen;
    c.D = headdim;
    c.R = rotary_dim;
    c.inv_freq = inv_freq;
    c.positions = positions;
    c.eps = eps;
    c.l2 = kind == SSM_QK_NORM_L2;
    c.interleaved = interleaved != 0;
    c.dtype = dtype;
    return hip_status(ssm::launch_qk_norm_fwd(c, reinterpret_cast<hipStream_t>(stream)), fn);
}

size_t ssm_qk_norm_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t headdim) {
    const int64_t most = int64_t{1} << 31;
    if (batch <= 0 || seqlen <= 0 || headdim < 1 || headdim > 256 || batch >= most || seqlen >= most / batch) return 0;
    return static_cast<size_t>(ssm::qk_norm_partial_rows(batch * seqlen) * 2 * headdim) * 4;
}

ssm_status_t ssm_qk_norm_bwd(const void* q, int64_t q_row, const void* k, int64_t k_row, const float* q_weight,
                             const float* k_weight, const float* inv_freq, const int32_t* positions,
                             const void* dq_out, int64_t dq_out_row, const void* dk_out, int64_t dk_out_row,
                             void* dq, int64_t dq_row, void* dk, int64_t dk_row, float* dq_weight,
                             float* dk_weight, void* workspace, size_t workspace_bytes, int64_t batch,
                             int64_t seqlen, int64_t nheads_q, int64_t nheads_k, int64_t headdim,
                             int64_t rotary_dim, int32_t interleaved, float eps, ssm_qk_norm_t kind,
                             ssm_dtype_t dtype, ssm_stream_t stream) {
    const char* fn = "ssm_qk_norm_bwd";
    ssm_status_t st = check_qk_norm_dims(fn, batch, seqlen, nheads_q, nheads_k, headdim, rotary_dim, inv_freq, eps, kind, dtype);
    if (st != SSM_OK) return st;
    const size_t es = esize(dtype);
    const int64_t rows = batch * seqlen;
    const bool work = rows > 0;
    st = check_ptrs(fn, {{"q", q, work, es},
                         {"k", k, work, es},
                         {"q_weight", q_weight, false, 4},
                         {"k_weight", k_weight, false, 4},
                         {"inv_freq", inv_freq, false, 4},
                         {"positions", positions, false, 4},
                         {"dq_out", dq_out, work, es},
                         {"dk_out", dk_out, work, es},
                         {"dq", dq, work, es},
                         {"dk", dk, work, es},
                         {"dq_weight", dq_weight, false, 4},
                         {"dk_weight", dk_weight, false, 4},
                         {"workspace", workspace, false, 4}});
    if (st == SSM_OK) st = check_row(fn, "q", q, q_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "k", k, k_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "dq_out", dq_out, dq_out_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "dk_out", dk_out, dk_out_row, rows, 0);
    if (st == SSM_OK) st = check_row(fn, "dq", dq, dq_row, rows, nheads_q * headdim);
    if (st == SSM_OK) st = check_row(fn, "dk", dk, dk_row, rows, nheads_k * headdim);
    if (st != SSM_OK) return st;
    const bool sums = dq_weight != nullptr || dk_weight != nullptr;
    if (work && sums) {
        const size_t need = ssm_qk_norm_bwd_workspace_size(batch, seqlen, headdim);
        if (workspace == nullptr || workspace_bytes < need)
            return fail(SSM_ERR_WORKSPACE, std::string(fn) + ": workspace missing or smaller than "
                                           "ssm_qk_norm_bwd_workspace_size");
    }
    if (!work && !sums) return ok();
    ssm::QkNormCall c{};
    c.x[0] = q;
    c.x[1] = k;
    c.x_row[0] = q_row;
    c.x_row[1] = k_row;
    c.dy[0] = dq_out;
    c.dy[1] = dk_out;
    c.dy_row[0] = dq_out_row;
    c.dy_row[1] = dk_out_row;
    c.out[0] = dq;
    c.out[1] = dk;
    c.out_row[0] = dq_row;
    c.out_row[1] = dk_row;
    c.w[0] = q_weight;
    c.w[1] = k_weight;
    c.dw[0] = dq_weight;
    c.dw[1] = dk_weight;
    c.partial = sums ? static_cast<float*>(workspace) : nullptr;
    c.heads[0] = nheads_q;
    c.heads[1] = nheads_k;
    c.tokens = rows;
    c.L = seqlen;
    c.D = headdim;
    c.R = rotary_dim;
    c.inv_freq = inv_freq;
    c.positions = positions;
    c.eps = eps;
    c.l2 = kind == SSM_QK_NORM_L2;
    c.interleaved = interleaved != 0;
    c.dtype = dtype;
    return hip_status(ssm::launch_qk_norm_bwd(c, reinterpret_cast<hipStream_t>(stream)), fn);
}

namespace {
ssm_status_t check_state_dims(const char* fn, int64_t batch, int64_t nheads, int64_t headdim,
                              int64_t dstate) {
    if (batch < 0) return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": negative batch");
    if (nheads < 1 || headdim < 1 || dstate < 1)
        return fail(SSM_ERR_INVALID_ARG, std::string(fn) + ": nheads, headdim, dstate must be >= 1");
    return SSM_OK;
}
}  // namespace

ssm_status_t ssm_state_stats_update(const float* final_state, int64_t batch, int64_t nheads,
                                    int64_t headdim, int64_t dstate, float beta, float* mean,
                                    float* var, ssm_stream_t stream) {
    const char* fn = "ssm_state_stats_update";
    ssm_status_t st = check_state_dims(fn, batch, nheads, headdim, dstate);
    if (st != SSM_OK) return st;
    if (!(beta == beta)) return fail(SSM_ERR_INVALID_ARG, "ssm_state_stats_update: beta is NaN");
    const bool rows = batch > 0;
    st = check_ptrs(fn, {{"final_state", final_state, rows, 4},
                         {"mean", mean, rows, 4},
                         {"var", var, rows, 4}});
    if (st != SSM_OK) return st;
    if (!rows) return ok();
    if (nheads > 0x7FFFFFFF)
        return fail(SSM_ERR_UNSUPPORTED, "ssm_state_stats_update: too many heads");
    return hip_status(ssm::launch_state_stats(final_state, batch, nheads, headdim * dstate,
                                              static_cast<double>(beta), mean, var,
                                              reinterpret_cast<hipStream_t>(stream)),
                      fn);
}

ssm_status_t ssm_initial_state_noise(float* out, int64_t batch, int64_t nheads, int64_t headdim,
                                     int64_t dstate, const float* mean, const float* var,
                                     float sigma, uint64_t seed, uint64_t offset,
                                     ssm_stream_t stream) {
    const char* fn = "ssm_initial_state_noise";
    ssm_status_t st = check_state_dims(fn, batch, nheads, headdim, dstate);
    if (st != SSM_OK) return st;
    if ((mean == nullptr) != (var == nullptr))
        return fail(SSM_ERR_INVALID_ARG, "ssm_initial_state_noise: give both mean and var, or neither");
    const bool rows = batch > 0;
    st = check_ptrs(fn, {{"out", out, rows, 4}, {"mean", mean, false, 4}, {"var", var, false, 4}});
    if (st != SSM_OK) return st;
    if (!rows) return ok();
    const int64_t n = batch * nheads * headdim * dstate;
    if ((n + 7) / 8 > static_cast<int64_t>(0xFFFFFFFFll) * 256)
        return fail(SSM_ERR_UNSUPPORTED, "ssm_initial_state_noise: tensor too large");
    return hip_status(ssm::launch_state_noise(out, n, nheads, headdim * dstate, mean, var, sigma,
                                              seed, offset, reinterpret_cast<hipStream_t>(stream)),
                      fn);
}

ssm_status_t ssm_state_reset(const void* src, void* dst, uint8_t* reset_mask, int64_t batch,
                             int64_t row_bytes, double p, uint64_t seed, uint64_t offset,
                             ssm_stream_t stream) {
    const char* fn = "ssm_state_reset";
    if (batch < 0 || row_bytes < 0 || (row_bytes & 1))
        return fail(SSM_ERR_INVALID_ARG, "ssm_state_reset: need batch >= 0 and an even row_bytes >= 0");
    if (!(p == p)) return fail(SSM_ERR_INVALID_ARG, "ssm_state_reset: p is NaN");
    const bool rows = batch > 0;
    ssm_status_t st = check_ptrs(fn, {{"src", src, rows && row_bytes > 0, 2},
                                      {"dst", dst, rows && row_bytes > 0, 2}});
    if (st != SSM_OK) return st;
    if (!rows) return ok();
    // threshold = floor(p 2^32), p clipped to [0, 1] (the scaling by 2^32 is exact)
    double t = std::floor((p < 0.0 ? 0.0 : p > 1.0 ? 1.0 : p) * 4294967296.0);
    const uint64_t threshold = static_cast<uint64_t>(t);
    const uintptr_t a = reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst);
    const int unit = ((a & 15) == 0 && row_bytes % 16 == 0) ? 16
                     : ((a & 3) == 0 && row_bytes % 4 == 0) ? 4 : 2;
    if (ssm::state_reset_blocks(batch, row_bytes, unit) > 0x7FFFFFFFll)
        return fail(SSM_ERR_UNSUPPORTED, "ssm_state_reset: tensor too large");
    return hip_status(ssm::launch_state_reset(src, dst, reset_mask, batch, row_bytes, unit,
                                              threshold, seed, offset,
                                              reinterpret_cast<hipStream_t>(stream)),
                      fn);
}

ssm_status_t ssm_stream_copy(const void* src, void* dst, int64_t bytes, ssm_stream_t stream) {
    const char* fn = "ssm_stream_copy";
    if (bytes < 0) return fail(SSM_ERR_INVALID_ARG, "ssm_stream_copy: need bytes >= 0");
    ssm_status_t st = check_ptrs(fn, {{"src", src, bytes > 0, 1}, {"dst", dst, bytes > 0, 1}});
    if (st != SSM_OK) return st;
    if (bytes == 0) return ok();
    const uintptr_t s0 = reinterpret_cast<uintptr_t>(src), d0 = reinterpret_cast<uintptr_t>(dst);
    if (s0 < d0 + static_cast<uintptr_t>(bytes) && d0 < s0 + static_cast<uintptr_t>(bytes))
        return fail(SSM_ERR_INVALID_ARG, "ssm_stream_copy: src and dst overlap");
    return hip_status(ssm::launch_stream_copy(src, dst, bytes, reinterpret_cast<hipStream_t>(stream)), fn);
}

ssm_status_t ssm_timing_enable(int enable) {
    std::lock_guard<std::mutex> lk(g_tmu);
    g_timing = enable != 0;
    return ok();
}

ssm_status_t ssm_timing_read(double* total_ms, int64_t* launches) {
    if (!total_ms || !launches) return fail(SSM_ERR_INVALID_ARG, "ssm_timing_read: NULL output");
    std::vector<EventPair> evs;
    {
        std::lock_guard<std::mutex> lk(g_tmu);
        evs.swap(g_events);
    }
    double sum = 0.0;
    hipError_t err = hipSuccess;
    for (auto& pr : evs) {
        float ms = 0.0f;
        hipError_t e = hipEventSynchronize(pr.e1);
        if (e == hipSuccess) e = hipEventElapsedTime(&ms, pr.e0, pr.e1);
        if (e != hipSuccess && err == hipSuccess) err = e;
        sum += ms;
    }
    {
        std::lock_guard<std::mutex> lk(g_tmu);
        g_spare.insert(g_spare.end(), evs.begin(), evs.end());
    }
    *total_ms = sum;
    *launches = static_cast<int64_t>(evs.size());
    return hip_status(err, "ssm_timing_read");
}

}  // extern "C"
