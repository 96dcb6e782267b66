// abi.cpp — the extern "C" entry points of libmdlstm: argument checks, workspace
// carving and kernel launches. Every check runs before the first launch, so a
// failing call writes nothing; errors never cross the ABI as exceptions.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <new>
#include <map>
#include <mutex>
#include <string>
#include <vector>

#include "../../include/mdlstm.h"
#include "kernels.h"
#include "leaky16.h"
#include "layout.h"

namespace mdl {
thread_local LaunchClock* t_launch_clock = nullptr;
}  // namespace mdl

namespace {

thread_local std::string g_err;

int fail(int code, const std::string& msg) {
    g_err = msg;
    return code;
}

int hip_fail(hipError_t e, const char* where) {
    return fail(MDL_EHIP, std::string(where) + ": " + hipGetErrorString(e));
}
int hip_fail(hipError_t e, const std::string& where) { return hip_fail(e, where.c_str()); }

const mdl::Layout& L_of(const mdl_layout* l) { return l->L; }

// ints of the workspace's flags region: the overlap's per-unit and per-task flags and its counters
int64_t nflags_of(const mdl::Layout& L) { return 4 * (int64_t)L.n + 8 * (int64_t)L.ngroups + mdl::kFlagTail; }
// ints of the workspace's forward flags region: the direction sum's overlap with the forward
int64_t nfflags_of(const mdl::Layout& L) { return 4 * (int64_t)L.n + 2 * (int64_t)L.nsum + mdl::kFlagTail; }

// the weight-gradient overlap: 1 on (default), 0 off, 2 on with no time to wait for any task (every task
// claimed beside the wavefront is given up and done after it); a stream (default priority) and fork / join
// events per device
std::atomic<int> g_overlap{1};
std::atomic<bool> g_scan_wait{true};
struct Side {
    hipStream_t s = nullptr;
    hipEvent_t fork = nullptr, join = nullptr;
    int ncu = 0;
};
constexpr int kMaxSideDevices = 64;
int side_of(Side*& out) {
    static std::mutex mu;
    static Side sides[kMaxSideDevices];
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e, "mdl_backward: current device");
    if (dev < 0 || dev >= kMaxSideDevices) return fail(MDL_EUNSUPPORTED, "mdl_backward: device index above 63");
    std::lock_guard<std::mutex> lk(mu);
    Side& sd = sides[dev];
    if (sd.s == nullptr) {
        Side n;
        if ((e = hipDeviceGetAttribute(&n.ncu, hipDeviceAttributeMultiprocessorCount, dev)) != hipSuccess ||
            (e = hipStreamCreateWithFlags(&n.s, hipStreamNonBlocking)) != hipSuccess ||
            (e = hipEventCreateWithFlags(&n.fork, hipEventDisableTiming)) != hipSuccess ||
            (e = hipEventCreateWithFlags(&n.join, hipEventDisableTiming)) != hipSuccess)
            return hip_fail(e, "mdl_backward: weight-gradient stream");
        sd = n;
    }
    out = &sd;
    return MDL_OK;
}

mdl::Dev make_dev(const mdl_layout* lay, const void* d_desc) {
    const mdl::Layout& L = L_of(lay);
    const uint8_t* b = static_cast<const uint8_t*>(d_desc);
    mdl::Dev D;
    D.rect = reinterpret_cast<const int32_t*>(b + L.off.rect);
    D.real = reinterpret_cast<const int32_t*>(b + L.off.real);
    D.flat_off = reinterpret_cast<const int64_t*>(b + L.off.flat_off);
    D.cell_off = reinterpret_cast<const int64_t*>(b + L.off.cell_off);
    D.units = reinterpret_cast<const int32_t*>(b + L.off.units);
    D.segs = reinterpret_cast<const int32_t*>(b + L.off.segs);
    D.groups = reinterpret_cast<const int32_t*>(b + L.off.groups);
    D.gorder = reinterpret_cast<const int32_t*>(b + L.off.gorder);
    D.dsum = reinterpret_cast<const int32_t*>(b + L.off.dsum);
    D.eid = reinterpret_cast<int32_t*>(const_cast<uint8_t*>(b + L.off.eid));
    D.border = const_cast<uint8_t*>(b + L.off.border);
    D.n = L.n;
    D.Hc = L.Hc;
    D.Wc = L.Wc;
    D.T = L.computed_cells;
    D.N = L.real_pixels;
    D.max_depth = L.max_depth;
    D.max_diag = L.max_diag;
    D.nsegs = L.nsegs;
    D.ngroups = L.ngroups;
    D.nsum = L.nsum;
    return D;
}

// LDS each workgroup of a launch beside a wavefront holds so that it cannot share a compute unit with one of the
// wavefront's workgroups (whose LDS is wave_lds, out of lmax per compute unit): those would then take the compute
// unit's issue slots from the wavefront's dependent chain, or, placed first, keep a wavefront workgroup waiting
size_t beside_lds_hold(size_t lmax, size_t wave_lds) { return wave_lds < lmax ? lmax - wave_lds + 256 : 0; }

int max_lds(size_t& out) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
    int v = 0;
    e = hipDeviceGetAttribute(&v, hipDeviceAttributeMaxSharedMemoryPerBlock, dev);
    if (e != hipSuccess) return hip_fail(e, "hipDeviceGetAttribute");
    out = (size_t)v;
    return MDL_OK;
}

int check_layer(const char* fn, const mdl_layout* layout, const void* d_desc, int32_t C, int32_t H, int32_t x_dtype) {
    if (!layout || !d_desc) return fail(MDL_EINVAL, std::string(fn) + ": null layout or descriptor");
    if (C < 1 || H < 1) return fail(MDL_EINVAL, std::string(fn) + ": need C >= 1 and H >= 1");
    if (x_dtype != MDL_F32 && x_dtype != MDL_BF16) return fail(MDL_EINVAL, std::string(fn) + ": unknown dtype");
    if (C > 1024 || H > 1024) return fail(MDL_EUNSUPPORTED, std::string(fn) + ": C or H above 1024");
    const mdl::Layout& L = L_of(layout);
    const int64_t P = (int64_t)L.Hc * L.Wc;
    if (P * 4 * std::max(H, C) >= (int64_t(1) << 40)) return fail(MDL_EOVERFLOW, std::string(fn) + ": canvas too large");
    return MDL_OK;
}

// ---- optional per-launch event timing ---------------------------------------------------------
struct TimedLaunch {
    std::string name;
    std::vector<hipEvent_t> ev;  // start, stop of each dispatch of the group, in launch order
};
bool g_timing = false;
std::string g_timing_only;  // empty: every group
std::mutex g_tmu;
std::vector<TimedLaunch> g_tlog;
std::vector<hipEvent_t> g_event_pool;

hipEvent_t take_event() {
    if (!g_event_pool.empty()) {
        hipEvent_t e = g_event_pool.back();
        g_event_pool.pop_back();
        return e;
    }
    hipEvent_t e = nullptr;
    if (hipEventCreate(&e) != hipSuccess) return nullptr;
    return e;
}

// While timing is on, installs itself as the thread's launch clock for one launcher call: each dispatch
// gets a start/stop event pair recorded by the dispatch itself, and the group's time runs from the first
// dispatch's start to the last one's stop.
class Timed : public mdl::LaunchClock {
  public:
    explicit Timed(const char* name) : name_(name) {
        if (!g_timing || (!g_timing_only.empty() && g_timing_only != name)) return;
        prev_ = mdl::t_launch_clock;
        mdl::t_launch_clock = this;
        on_ = true;
    }
    ~Timed() override {
        if (!on_) return;
        mdl::t_launch_clock = prev_;
        if (ev_.empty()) return;
        std::lock_guard<std::mutex> lk(g_tmu);
        g_tlog.push_back({name_, std::move(ev_)});
    }
    void events(hipEvent_t* start, hipEvent_t* stop) override {
        std::lock_guard<std::mutex> lk(g_tmu);
        hipEvent_t a = take_event(), b = take_event();
        if (!a || !b) {
            if (a) g_event_pool.push_back(a);
            if (b) g_event_pool.push_back(b);
            return;
        }
        ev_.push_back(a);
        ev_.push_back(b);
        *start = a;
        *stop = b;
    }

  private:
    const char* name_;
    bool on_ = false;
    mdl::LaunchClock* prev_ = nullptr;
    std::vector<hipEvent_t> ev_;
};

#define GUARD_BEGIN try {
#define GUARD_END                                                      \
    }                                                                  \
    catch (const std::bad_alloc&) { return fail(MDL_ENOMEM, "out of host memory"); } \
    catch (...) { return fail(MDL_EINVAL, "unexpected internal error"); }

}  // namespace

extern "C" {

int mdl_pack(const int32_t* heights, const int32_t* widths, int32_t n, int32_t canvas_w_min, int32_t sep,
             int32_t mode, mdl_layout** out) {
    GUARD_BEGIN
    if (!out) return fail(MDL_EINVAL, "mdl_pack: null output pointer");
    *out = nullptr;
    mdl_layout* lay = new (std::nothrow) mdl_layout;
    if (!lay) return fail(MDL_ENOMEM, "mdl_pack: out of host memory");
    std::string err;
    const int rc = mdl::build_layout(heights, widths, n, canvas_w_min, sep, mode, lay->L, err);
    if (rc != MDL_OK) {
        delete lay;
        return fail(rc, err);
    }
    *out = lay;
    return MDL_OK;
    GUARD_END
}

int mdl_pack_level(const mdl_layout* lk, int32_t kh, int32_t kw, int32_t canvas_w_min, int32_t sep, int32_t mode,
                   mdl_layout** out) {
    GUARD_BEGIN
    if (!out) return fail(MDL_EINVAL, "mdl_pack_level: null output pointer");
    *out = nullptr;
    if (!lk) return fail(MDL_EINVAL, "mdl_pack_level: null layout");
    if (kh < 1 || kw < 1) return fail(MDL_EINVAL, "mdl_pack_level: block sizes must be positive");
    const mdl::Layout& A = L_of(lk);
    // the block-strided convolution covers each example with ceil(h / kh) x ceil(w / kw) blocks, the last
    // row and column of blocks padded with zeros
    std::vector<int32_t> hs(A.n), ws(A.n);
    for (int e = 0; e < A.n; ++e) {
        hs[e] = (A.real[4 * e + 2] + kh - 1) / kh;
        ws[e] = (A.real[4 * e + 3] + kw - 1) / kw;
    }
    return mdl_pack(hs.data(), ws.data(), A.n, canvas_w_min, sep, mode, out);
    GUARD_END
}

void mdl_layout_free(mdl_layout* layout) { delete layout; }

int mdl_layout_info(const mdl_layout* layout, int64_t* info) {
    if (!layout || !info) return fail(MDL_EINVAL, "mdl_layout_info: null argument");
    const mdl::Layout& L = L_of(layout);
    info[MDL_INFO_N] = L.n;
    info[MDL_INFO_CANVAS_H] = L.Hc;
    info[MDL_INFO_CANVAS_W] = L.Wc;
    info[MDL_INFO_ROWS] = (int64_t)L.rows.size();
    info[MDL_INFO_REAL_PIXELS] = L.real_pixels;
    info[MDL_INFO_COMPUTED_CELLS] = L.computed_cells;
    info[MDL_INFO_MAX_DEPTH] = L.max_depth;
    info[MDL_INFO_MAX_DIAG] = L.max_diag;
    info[MDL_INFO_MODE] = L.mode;
    info[MDL_INFO_WG_GROUPS] = L.ngroups;
    return MDL_OK;
}

int mdl_layout_rects(const mdl_layout* layout, int32_t* rects, int32_t* real) {
    if (!layout) return fail(MDL_EINVAL, "mdl_layout_rects: null layout");
    const mdl::Layout& L = L_of(layout);
    if (rects) std::memcpy(rects, L.rect.data(), sizeof(int32_t) * 4 * L.n);
    if (real) std::memcpy(real, L.real.data(), sizeof(int32_t) * 4 * L.n);
    return MDL_OK;
}

int mdl_layout_rows(const mdl_layout* layout, int32_t* row_start, int32_t* row_examples) {
    if (!layout || !row_start || !row_examples) return fail(MDL_EINVAL, "mdl_layout_rows: null argument");
    const mdl::Layout& L = L_of(layout);
    int32_t k = 0;
    for (size_t r = 0; r < L.rows.size(); ++r) {
        row_start[r] = k;
        for (int32_t e : L.rows[r]) row_examples[k++] = e;
    }
    row_start[L.rows.size()] = k;
    return MDL_OK;
}

int mdl_layout_units(const mdl_layout* layout, int32_t* units, size_t* desc_offset) {
    if (!layout || !units || !desc_offset) return fail(MDL_EINVAL, "mdl_layout_units: null argument");
    const mdl::Layout& L = L_of(layout);
    std::copy(L.units.begin(), L.units.end(), units);
    *desc_offset = L.off.units;
    return MDL_OK;
}

int mdl_layout_maps(const mdl_layout* layout, int32_t* eid, uint8_t* border) {
    if (!layout) return fail(MDL_EINVAL, "mdl_layout_maps: null layout");
    const mdl::Layout& L = L_of(layout);
    if (eid) std::memcpy(eid, L.eid.data(), sizeof(int32_t) * L.eid.size());
    if (border) std::memcpy(border, L.border.data(), L.border.size());
    return MDL_OK;
}

int mdl_layout_device_size(const mdl_layout* layout, size_t* bytes, size_t* eid_offset, size_t* border_offset) {
    if (!layout || !bytes) return fail(MDL_EINVAL, "mdl_layout_device_size: null argument");
    const mdl::Layout& L = L_of(layout);
    *bytes = L.off.total;
    if (eid_offset) *eid_offset = L.off.eid;
    if (border_offset) *border_offset = L.off.border;
    return MDL_OK;
}

int mdl_layout_upload(const mdl_layout* layout, void* d_desc, size_t bytes, void* stream) {
    GUARD_BEGIN
    if (!layout || !d_desc) return fail(MDL_EINVAL, "mdl_layout_upload: null argument");
    const mdl::Layout& L = L_of(layout);
    if (bytes < L.off.total) return fail(MDL_ESIZE, "mdl_layout_upload: descriptor buffer too small");
    if (reinterpret_cast<uintptr_t>(d_desc) % 8) return fail(MDL_EINVAL, "mdl_layout_upload: descriptor not 8-byte aligned");
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e = hipMemcpyAsync(d_desc, L.host_desc.data(), L.host_desc.size(), hipMemcpyHostToDevice, st);
    if (e != hipSuccess) return hip_fail(e, "mdl_layout_upload: copy");
    {
        Timed t("build_maps");
        e = mdl::launch_build_maps(make_dev(layout, d_desc), st);
    }
    if (e != hipSuccess) return hip_fail(e, "mdl_layout_upload: map kernels");
    e = hipStreamSynchronize(st);
    if (e != hipSuccess) return hip_fail(e, "mdl_layout_upload: synchronize");
    return MDL_OK;
    GUARD_END
}

int mdl_workspace_size(const mdl_layout* layout, int32_t C, int32_t H, size_t* bytes) {
    if (!layout || !bytes) return fail(MDL_EINVAL, "mdl_workspace_size: null argument");
    if (C < 1 || H < 1) return fail(MDL_EINVAL, "mdl_workspace_size: need C >= 1 and H >= 1");
    *bytes = mdl::ws_layout(L_of(layout).computed_cells, L_of(layout).nparts(), C, H, nflags_of(L_of(layout)), nfflags_of(L_of(layout))).total;
    return MDL_OK;
}

int mdl_scatter(const mdl_layout* layout, const void* d_desc, const void* x_flat, int32_t C, int32_t dtype,
                void* x_canvas, void* stream) {
    GUARD_BEGIN
    int rc = check_layer("mdl_scatter", layout, d_desc, C, 1, dtype);
    if (rc) return rc;
    if (!x_flat || !x_canvas) return fail(MDL_EINVAL, "mdl_scatter: null tensor");
    hipError_t e;
    {
        Timed t("scatter");
        e = mdl::launch_scatter(make_dev(layout, d_desc), x_flat, C, dtype, x_canvas, static_cast<hipStream_t>(stream));
    }
    if (e != hipSuccess) return hip_fail(e, "mdl_scatter");
    return MDL_OK;
    GUARD_END
}

// The kernels address device tensors through buffer descriptors with 32-bit byte ranges and offsets.
// The wavefront kernels take one direction's h plane and the canvas input each as one range and send a
// masked lane 2^30 bytes past its start; the gate stash is addressed one example at a time. The
// software-pipelined weight-gradient kernel takes one direction's h plane and gate gradients per range.
static int check_extent(const char* fn, const mdl::Layout& L, int C, int H, int x_dtype, bool backward) {
    const int64_t plane = (int64_t)L.Hc * L.Wc * H * 4;
    const int64_t xbytes = (int64_t)L.Hc * L.Wc * C * (x_dtype == MDL_BF16 ? 2 : 4);
    const int64_t dabytes = L.computed_cells * 5 * (int64_t)H * 4;  // one direction
    const int64_t lim = (int64_t(1) << 31) - 16;
    if (plane > (int64_t(1) << 30) || xbytes > (int64_t(1) << 30))
        return fail(MDL_EUNSUPPORTED, std::string(fn) + ": one direction's h plane or the canvas input above 1 GiB");
    if (backward && dabytes >= lim)
        return fail(MDL_EUNSUPPORTED, std::string(fn) + ": one direction's gate gradients above 2 GiB");
    // The wavefront kernels address one example's stash and gate gradients (at most 16 H bytes per cell) through
    // a per-example buffer range and park the accesses of idle lanes at byte offset 2^30, which must lie past
    // that range.
    int64_t cells = 0;
    for (int e = 0; e < L.n; ++e) cells = std::max<int64_t>(cells, (int64_t)L.rect[4 * e + 2] * L.rect[4 * e + 3]);
    if (cells * 16 * H > (int64_t(1) << 30))
        return fail(MDL_EUNSUPPORTED, std::string(fn) + ": one example's cells x 16 H bytes above 1 GiB");
    return MDL_OK;
}

static int check_cell(const char* fn, int32_t cell, const void* Vl, const void* Vu) {
    if (cell == MDL_CELL_MDLSTM) {
        if (Vl || Vu) return fail(MDL_EINVAL, std::string(fn) + ": memory-state projections given with the MDLSTM cell");
        return MDL_OK;
    }
    if (cell == MDL_CELL_LEAKY_LP) {
        if (!Vl || !Vu) return fail(MDL_EINVAL, std::string(fn) + ": the Leaky LP cell needs its memory-state projections");
        return MDL_OK;
    }
    return fail(MDL_EINVAL, std::string(fn) + ": unknown cell");
}

// The forward wavefront of mdl_forward and, when y_flat is given, the direction sum of mdl_dirsum_unpack.
// The sum overlaps the wavefront when its units leave at least half of the compute units free (f16 path,
// chunked sum supported): each unit flags itself when its h plane is stored, persistent workgroups on the
// library's second stream take the sum's chunks (in the order their examples finish) once all four of an
// example's units are done, and the launch after the wavefront takes the rest; every chunk runs the same code.
static int forward_impl(const char* fn, const mdl_layout* layout, const void* d_desc, const void* x_canvas,
                        int32_t x_dtype, int32_t C, int32_t H, int32_t cell, const float* Wx, const float* Ul,
                        const float* Uu, const float* b, const float* Vl, const float* Vu, float* h_dirs,
                        float* y_flat, void* ws, size_t ws_bytes, void* stream) {
    const std::string F(fn);
    int rc = check_layer(fn, layout, d_desc, C, H, x_dtype);
    if (rc) return rc;
    if ((rc = check_cell(fn, cell, Vl, Vu))) return rc;
    if (!x_canvas || !Wx || !Ul || !Uu || !b || !h_dirs || !ws) return fail(MDL_EINVAL, F + ": null tensor");
    const mdl::Layout& L = L_of(layout);
    const mdl::WsLayout W = mdl::ws_layout(L.computed_cells, L.nparts(), C, H, nflags_of(L), nfflags_of(L));
    if (ws_bytes < W.total) return fail(MDL_ESIZE, F + ": workspace smaller than mdl_workspace_size");
    if ((rc = check_extent(fn, L, C, H, x_dtype, false))) return rc;
    const mdl::Dev D = make_dev(layout, d_desc);
    hipStream_t st = static_cast<hipStream_t>(stream);
    uint8_t* wsb = static_cast<uint8_t*>(ws);
    float* stash = reinterpret_cast<float*>(wsb + W.stash);
    hipError_t e = hipSuccess;
    // the direction sum after the wavefront (when asked for and not overlapped)
    auto dirsum_after = [&]() -> int {
        if (!y_flat) return MDL_OK;
        Timed t("dirsum");
        const hipError_t e2 = mdl::launch_dirsum(D, h_dirs, H, y_flat, st);
        return e2 == hipSuccess ? MDL_OK : hip_fail(e2, F + ": direction sum");
    };
    if (cell == MDL_CELL_LEAKY_LP) {
        if (!mdl::leaky_supported(H, C, L.max_diag))
            return fail(MDL_EUNSUPPORTED, F + ": the Leaky LP cell runs for H in {4, 8, 16, 32}, C <= 16 and "
                                              "a widest diagonal of at most 64 cells (32 at H = 32)");
        size_t lmax = 0;
        if ((rc = max_lds(lmax))) return rc;
        if (mdl::leaky_fwd_lds(H, L.max_diag) > lmax) return fail(MDL_EUNSUPPORTED, F + ": diagonal state exceeds LDS");
        {
            Timed t("zero_fill");
            e = mdl::launch_zero_outside(D, h_dirs, H, 4, st);
        }
        if (e != hipSuccess) return hip_fail(e, F + ": zero fill");
        {
            Timed t("fwd_wavefront");
            e = mdl::launch_fwd_leaky(D, x_canvas, x_dtype, C, H, Wx, b, Ul, Uu, Vl, Vu, stash, h_dirs, st);
        }
        if (e != hipSuccess) return hip_fail(e, F + ": wavefront");
        return dirsum_after();
    }
    // small hidden sizes: vector-ALU wavefront; instantiated matrix-core shapes: f16 wavefront; both with
    // the projection fused. Otherwise the projection as its own GEMM and the general fp32 wavefront.
    const bool small = mdl::small_fwd_supported(H, C, x_dtype, L.max_diag);
    const bool fused = !small && mdl::fwd16_supported(H, C, x_dtype, L.max_diag);
    if (!small && !fused && (int64_t)L.max_diag * H > mdl::chain_max_items())
        return fail(MDL_EUNSUPPORTED, F + ": widest diagonal x H exceeds the wavefront kernel's items");
    size_t lmax = 0;
    if ((rc = max_lds(lmax))) return rc;
    const size_t need = small ? mdl::small_fwd_lds(H, L.max_diag)
                              : (fused ? mdl::fwd16_lds(H, C, x_dtype, L.max_diag) : mdl::fwd_chain_lds(H, L.max_diag));
    if (need > lmax) return fail(MDL_EUNSUPPORTED, F + ": recurrent weights and diagonal state exceed LDS");
    float* Z = reinterpret_cast<float*>(wsb + W.zda);
    if (!fused) {  // the f16 forward clears h outside the computed regions itself, in its smallest units' tail
        Timed t("zero_fill");
        e = mdl::launch_zero_outside(D, h_dirs, H, 4, st);
    }
    if (e != hipSuccess) return hip_fail(e, F + ": zero fill");
    Side* side = nullptr;
    int ov_wg = 0;
    const int ov_mode = g_overlap.load();
    if (fused && y_flat && ov_mode != 0 && mdl::dirsum_chunked_supported(D, h_dirs, H, y_flat)) {
        if ((rc = side_of(side))) return rc;
        const int free_cu = side->ncu - 4 * L.n;
        if (2 * free_cu >= side->ncu) ov_wg = std::min(free_cu, (int)L.nsum);
    }
    mdl::OverlapFlags Fl{};
    if (ov_wg > 0) {
        int32_t* fl = reinterpret_cast<int32_t*>(wsb + W.fflags);
        Fl.done = fl;
        Fl.taken = fl + 4 * L.n;
        Fl.abandoned = Fl.taken + L.nsum;
        Fl.queue = Fl.abandoned + L.nsum;
        Fl.stop = Fl.queue + 1;
        Fl.nab = Fl.queue + 2;
        Fl.abq = Fl.queue + 3;
        if ((e = mdl::launch_fill_i32(fl, nfflags_of(L), 0, st)) != hipSuccess)
            return hip_fail(e, F + ": overlap flags");
        if ((e = hipEventRecord(side->fork, st)) != hipSuccess || (e = hipStreamWaitEvent(side->s, side->fork, 0)) != hipSuccess)
            return hip_fail(e, F + ": fork to the library's stream");
    }
    if (small) {
        Timed t("fwd_wavefront");
        e = mdl::launch_fwd_small(D, x_canvas, x_dtype, C, H, Wx, b, Ul, Uu, stash, h_dirs, st);
    } else if (fused) {
        Timed t("fwd_wavefront");
        e = mdl::launch_fwd16(D, x_canvas, x_dtype, C, H, Wx, b, Ul, Uu, stash, h_dirs, ov_wg > 0 ? Fl.done : nullptr,
                              st);
    } else {
        {
            Timed t("projection");
            e = mdl::launch_projection(D, x_canvas, x_dtype, C, H, Wx, b, Z, st);
        }
        if (e != hipSuccess) return hip_fail(e, F + ": projection");
        Timed t("fwd_wavefront");
        e = mdl::launch_fwd_chain(D, H, Ul, Uu, Z, stash, h_dirs, st);
    }
    if (e != hipSuccess) return hip_fail(e, F + ": wavefront");
    if (ov_wg == 0) return dirsum_after();
    // each wait at most ~2^15 clock cycles per dependent step of the layout, at least 2^26 cycles
    const long long budget = ov_mode == 2 ? 0 : std::max<long long>(1ll << 26, (long long)L.max_depth << 15);
    {
        Timed t("dirsum_overlap");
        e = mdl::launch_dirsum_claim(D, h_dirs, H, y_flat, Fl, mdl::kClaimBeside, ov_wg, budget,
                                     beside_lds_hold(lmax, need), side->s);
    }
    if (e != hipSuccess) return hip_fail(e, F + ": direction sum beside the wavefront");
    if ((e = hipEventRecord(side->join, side->s)) != hipSuccess) return hip_fail(e, F + ": library's stream");
    {
        Timed t("dirsum");
        e = mdl::launch_dirsum_claim(D, h_dirs, H, y_flat, Fl, mdl::kClaimDrain, 0, 0, 0, st);
        if (e == hipSuccess && (e = hipStreamWaitEvent(st, side->join, 0)) == hipSuccess)
            e = mdl::launch_dirsum_claim(D, h_dirs, H, y_flat, Fl, mdl::kClaimAbandoned, 16, 0, 0, st);
    }
    if (e != hipSuccess) return hip_fail(e, F + ": direction sum");
    return MDL_OK;
}

int mdl_forward(const mdl_layout* layout, const void* d_desc, const void* x_canvas, int32_t x_dtype, int32_t C,
                int32_t H, int32_t cell, const float* Wx, const float* Ul, const float* Uu, const float* b,
                const float* Vl, const float* Vu, float* h_dirs, void* ws, size_t ws_bytes, void* stream) {
    GUARD_BEGIN
    return forward_impl("mdl_forward", layout, d_desc, x_canvas, x_dtype, C, H, cell, Wx, Ul, Uu, b, Vl, Vu, h_dirs,
                        nullptr, ws, ws_bytes, stream);
    GUARD_END
}

int mdl_forward_dirsum(const mdl_layout* layout, const void* d_desc, const void* x_canvas, int32_t x_dtype,
                       int32_t C, int32_t H, int32_t cell, const float* Wx, const float* Ul, const float* Uu,
                       const float* b, const float* Vl, const float* Vu, float* h_dirs, float* y_flat, void* ws,
                       size_t ws_bytes, void* stream) {
    GUARD_BEGIN
    if (!y_flat) return fail(MDL_EINVAL, "mdl_forward_dirsum: null tensor");
    return forward_impl("mdl_forward_dirsum", layout, d_desc, x_canvas, x_dtype, C, H, cell, Wx, Ul, Uu, b, Vl, Vu,
                        h_dirs, y_flat, ws, ws_bytes, stream);
    GUARD_END
}

static size_t skew_dcb_offset(const mdl::WsLayout& W) { return (W.total + 255) & ~size_t(255); }

int mdl_skewed_workspace_size(const mdl_layout* layout, int32_t C, int32_t H, size_t* bytes) {
    if (!layout || !bytes) return fail(MDL_EINVAL, "mdl_skewed_workspace_size: null argument");
    if (C < 1 || H < 1) return fail(MDL_EINVAL, "mdl_skewed_workspace_size: need C >= 1 and H >= 1");
    const mdl::Layout& L = L_of(layout);
    const mdl::WsLayout W = mdl::ws_layout(L.computed_cells, L.nparts(), C, H, nflags_of(L), nfflags_of(L));
    *bytes = skew_dcb_offset(W) + sizeof(float) * 4 * (size_t)L.computed_cells * 2 * H;
    return MDL_OK;
}

int mdl_forward_skewed(const mdl_layout* layout, const void* d_desc, const void* x_canvas, int32_t x_dtype,
                       int32_t C, int32_t H, const float* Wx, const float* Ul, const float* Uu, const float* b,
                       float* h_dirs, void* ws, size_t ws_bytes, void* stream) {
    GUARD_BEGIN
    int rc = check_layer("mdl_forward_skewed", layout, d_desc, C, H, x_dtype);
    if (rc) return rc;
    if (!x_canvas || !Wx || !Ul || !Uu || !b || !h_dirs || !ws)
        return fail(MDL_EINVAL, "mdl_forward_skewed: null tensor");
    if (!mdl::skew_supported(H)) return fail(MDL_EUNSUPPORTED, "mdl_forward_skewed: runs for H in {4, 16}");
    const mdl::Layout& L = L_of(layout);
    size_t need = 0;
    mdl_skewed_workspace_size(layout, C, H, &need);
    if (ws_bytes < need) return fail(MDL_ESIZE, "mdl_forward_skewed: workspace smaller than mdl_skewed_workspace_size");
    if ((rc = check_extent("mdl_forward_skewed", L, C, H, x_dtype, true))) return rc;
    const mdl::WsLayout W = mdl::ws_layout(L.computed_cells, L.nparts(), C, H, nflags_of(L), nfflags_of(L));
    const mdl::Dev D = make_dev(layout, d_desc);
    hipStream_t st = static_cast<hipStream_t>(stream);
    uint8_t* wsb = static_cast<uint8_t*>(ws);
    float* Z = reinterpret_cast<float*>(wsb + W.zda);
    float* stash = reinterpret_cast<float*>(wsb + W.stash);
    hipError_t e;
    {
        Timed t("zero_fill");
        e = mdl::launch_zero_outside(D, h_dirs, H, 4, st);
    }
    if (e != hipSuccess) return hip_fail(e, "mdl_forward_skewed: zero fill");
    {
        Timed t("projection");
        e = mdl::launch_projection(D, x_canvas, x_dtype, C, H, Wx, b, Z, st);
    }
    if (e != hipSuccess) return hip_fail(e, "mdl_forward_skewed: projection");
    {
        Timed t("fwd_skewed_columns");
        e = mdl::launch_skew_fwd(D, H, Ul, Uu, Z, stash, h_dirs, st);
    }
    if (e != hipSuccess) return hip_fail(e, "mdl_forward_skewed: column steps");
    return MDL_OK;
    GUARD_END
}

int mdl_backward_skewed(const mdl_layout* layout, const void* d_desc, const void* x_canvas, int32_t x_dtype,
                        int32_t C, int32_t H, const float* Wx, const float* Ul, const float* Uu, const float* h_dirs,
                        const float* dy_flat, const float* dh_dirs, float* dx_flat, float* dx_canvas, float* dWx,
                        float* dUl, float* dUu, float* db, void* ws, size_t ws_bytes, void* stream) {
    GUARD_BEGIN
    int rc = check_layer("mdl_backward_skewed", layout, d_desc, C, H, x_dtype);
    if (rc) return rc;
    if (!x_canvas || !Wx || !Ul || !Uu || !h_dirs || !ws || !dWx || !dUl || !dUu || !db)
        return fail(MDL_EINVAL, "mdl_backward_skewed: null tensor");
    if ((dy_flat == nullptr) == (dh_dirs == nullptr))
        return fail(MDL_EINVAL, "mdl_backward_skewed: pass exactly one of dy_flat and dh_dirs");
    if (!mdl::skew_supported(H)) return fail(MDL_EUNSUPPORTED, "mdl_backward_skewed: runs for H in {4, 16}");
    const mdl::Layout& L = L_of(layout);
    size_t need = 0;
    mdl_skewed_workspace_size(layout, C, H, &need);
    if (ws_bytes < need)
        return fail(MDL_ESIZE, "mdl_backward_skewed: workspace smaller than mdl_skewed_workspace_size");
    if ((rc = check_extent("mdl_backward_skewed", L, C, H, x_dtype, true))) return rc;
    const bool wg2 = mdl::wgrad2_supported(C, H, x_dtype);
    size_t lmax = 0;
    if ((rc = max_lds(lmax))) return rc;
    if ((wg2 ? mdl::wgrad2_lds_bytes(C, H, x_dtype) : mdl::wgrad_lds_bytes(C, H)) > lmax)
        return fail(MDL_EUNSUPPORTED, "mdl_backward_skewed: weight-gradient tile exceeds LDS");
    const mdl::WsLayout W = mdl::ws_layout(L.computed_cells, L.nparts(), C, H, nflags_of(L), nfflags_of(L));
    const mdl::Dev D = make_dev(layout, d_desc);
    hipStream_t st = static_cast<hipStream_t>(stream);
    uint8_t* wsb = static_cast<uint8_t*>(ws);
    float* dA = reinterpret_cast<float*>(wsb + W.zda);
    const float* stash = reinterpret_cast<const float*>(wsb + W.stash);
    float* part = reinterpret_cast<float*>(wsb + W.part);
    float* dxp = reinterpret_cast<float*>(wsb + W.dxp);
    float* dcb = reinterpret_cast<float*>(wsb + skew_dcb_offset(W));
    hipError_t e;
    {
        Timed t("bwd_skewed_columns");
        e = mdl::launch_skew_bwd(D, H, Ul, Uu, stash, dy_flat, dh_dirs, dA, dcb, st);
    }
    if (e != hipSuccess) return hip_fail(e, "mdl_backward_skewed: column steps");
    if (dx_canvas) {
        Timed t("zero_fill");
        e = mdl::launch_zero_outside(D, dx_canvas, C, 1, st);
        if (e != hipSuccess) return hip_fail(e, "mdl_backward_skewed: zero fill");
    }
    {
        Timed t("wgrad");
        e = mdl::launch_wgrad(D, x_canvas, x_dtype, C, H, h_dirs, dA, Wx, part, dxp, dWx, dUl, dUu, db, dx_flat,
                              dx_canvas, st);
    }
    if (e != hipSuccess) return hip_fail(e, "mdl_backward_skewed: weight and input gradients");
    return MDL_OK;
    GUARD_END
}

int mdl_dirsum_unpack(const mdl_layout* layout, const void* d_desc, const float* h_dirs, int32_t H, float* y_flat,
                      void* stream) {
    GUARD_BEGIN
    int rc = check_layer("mdl_dirsum_unpack", layout, d_desc, 1, H, MDL_F32);
    if (rc) return rc;
    if (!h_dirs || !y_flat) return fail(MDL_EINVAL, "mdl_dirsum_unpack: null tensor");
    hipError_t e;
    {
        Timed t("dirsum");
        e = mdl::launch_dirsum(make_dev(layout, d_desc), h_dirs, H, y_flat, static_cast<hipStream_t>(stream));
    }
    if (e != hipSuccess) return hip_fail(e, "mdl_dirsum_unpack");
    return MDL_OK;
    GUARD_END
}

int mdl_backward(const mdl_layout* layout, const void* d_desc, const void* x_canvas, int32_t x_dtype, int32_t C,
                 int32_t H, int32_t cell, const float* Wx, const float* Ul, const float* Uu, const float* Vl,
                 const float* Vu, const float* h_dirs, const float* dy_flat, const float* dh_dirs, float* dx_flat,
                 float* dx_canvas, float* dWx, float* dUl, float* dUu, float* db, float* dVl, float* dVu, void* ws,
                 size_t ws_bytes, void* stream) {
    GUARD_BEGIN
    int rc = check_layer("mdl_backward", layout, d_desc, C, H, x_dtype);
    if (rc) return rc;
    if ((rc = check_cell("mdl_backward", cell, Vl, Vu))) return rc;
    const bool lk = cell == MDL_CELL_LEAKY_LP;
    if (lk != (dVl != nullptr) || lk != (dVu != nullptr))
        return fail(MDL_EINVAL, "mdl_backward: dVl and dVu go with the Leaky LP cell, and only with it");
    if (!x_canvas || !Wx || !Ul || !Uu || !h_dirs || !ws) return fail(MDL_EINVAL, "mdl_backward: null tensor");
    if (!dWx || !dUl || !dUu || !db) return fail(MDL_EINVAL, "mdl_backward: null weight-gradient output");
    if ((dy_flat == nullptr) == (dh_dirs == nullptr))
        return fail(MDL_EINVAL, "mdl_backward: pass exactly one of dy_flat and dh_dirs");
    const mdl::Layout& L = L_of(layout);
    const mdl::WsLayout W = mdl::ws_layout(L.computed_cells, L.nparts(), C, H, nflags_of(L), nfflags_of(L));
    if (ws_bytes < W.total) return fail(MDL_ESIZE, "mdl_backward: workspace smaller than mdl_workspace_size");
    if (lk && !mdl::leaky_supported(H, C, L.max_diag))
        return fail(MDL_EUNSUPPORTED, "mdl_backward: the Leaky LP cell runs for H in {4, 8, 16, 32}, C <= 16 and a "
                                      "widest diagonal of at most 64 cells (32 at H = 32)");
    if (!lk && !mdl::small_bwd_supported(H, L.max_diag) && !mdl::bwd16_supported(H, L.max_diag) &&
        !mdl::chain_uses_mfma(H, L.max_diag) &&
        (int64_t)L.max_diag * H > mdl::chain_max_items())
        return fail(MDL_EUNSUPPORTED, "mdl_backward: widest diagonal x H exceeds the wavefront kernel's items");
    const bool wg2 = mdl::wgrad2_supported(C, H, x_dtype);
    if ((rc = check_extent("mdl_backward", L, C, H, x_dtype, true))) return rc;
    size_t lmax = 0;
    if ((rc = max_lds(lmax))) return rc;
    if ((lk ? mdl::leaky_bwd_lds(H, L.max_diag) : mdl::bwd_chain_lds(H, L.max_diag)) > lmax)
        return fail(MDL_EUNSUPPORTED, "mdl_backward: recurrent weights and diagonal state exceed LDS");
    if ((wg2 ? mdl::wgrad2_lds_bytes(C, H, x_dtype) : mdl::wgrad_lds_bytes(C, H)) > lmax)
        return fail(MDL_EUNSUPPORTED, "mdl_backward: weight-gradient tile exceeds LDS");
    const mdl::Dev D = make_dev(layout, d_desc);
    hipStream_t st = static_cast<hipStream_t>(stream);
    uint8_t* wsb = static_cast<uint8_t*>(ws);
    float* dA = reinterpret_cast<float*>(wsb + W.zda);
    const float* stash = reinterpret_cast<const float*>(wsb + W.stash);
    float* part = reinterpret_cast<float*>(wsb + W.part);
    float* dxp = reinterpret_cast<float*>(wsb + W.dxp);
    const bool want_dx = dx_flat != nullptr || dx_canvas != nullptr;
    hipError_t e;
    // The weight gradient overlaps the reverse wavefront when the wavefront's units leave at least half of
    // the compute units free: each unit flags itself when done, and persistent workgroups on a second
    // stream (one per free compute unit, so the wavefront's units always find room) take the weight-gradient
    // tasks (one direction of one group) from a claim queue, in the order their units finish, once those
    // units are done. The launch after the wavefront takes the rest of the queue on every compute unit while
    // they finish their last tasks; a third launch, after both, does any task given up beside the wavefront
    // for want of time. Each task is computed by the same code either way.
    Side* side = nullptr;
    int ov_wg = 0;
    const int ov_mode = g_overlap.load();
    // (the Leaky-LP cell's gate gradients have the plain cell's layout: the same tasks, once its 16-bit reverse
    // wavefront flags its units)
    if (ov_mode != 0 && wg2 && (lk ? mdl::leaky16_used(H, L.max_diag) : mdl::bwd16_supported(H, L.max_diag))) {
        if ((rc = side_of(side))) return rc;
        const int free_cu = side->ncu - 4 * L.n;
        if (2 * free_cu >= side->ncu) ov_wg = std::min(free_cu, 4 * (int)L.ngroups);
    }
    mdl::OverlapFlags F{};
    if (ov_wg > 0) {
        int32_t* fl = reinterpret_cast<int32_t*>(wsb + W.flags);
        F.done = fl;
        F.taken = fl + 4 * L.n;
        F.abandoned = F.taken + 4 * L.ngroups;
        F.queue = F.abandoned + 4 * L.ngroups;
        F.stop = F.queue + 1;
        F.nab = F.queue + 2;
        F.abq = F.queue + 3;
        if ((e = mdl::launch_fill_i32(fl, nflags_of(L), 0, st)) != hipSuccess)
            return hip_fail(e, "mdl_backward: overlap counters");
        if ((e = hipEventRecord(side->fork, st)) != hipSuccess || (e = hipStreamWaitEvent(side->s, side->fork, 0)) != hipSuccess)
            return hip_fail(e, "mdl_backward: fork to the weight-gradient stream");
    }
    {
        Timed t("bwd_wavefront");
        e = lk ? (ov_wg > 0 ? mdl::launch_bwd_leaky16(D, H, Ul, Uu, Vl, Vu, stash, dy_flat, dh_dirs, dA, F.done, st)
                            : mdl::launch_bwd_leaky(D, H, Ul, Uu, Vl, Vu, stash, dy_flat, dh_dirs, dA, st))
           : ov_wg > 0 ? mdl::launch_bwd16(D, H, Ul, Uu, stash, dy_flat, dh_dirs, dA, F.done, st)
                       : mdl::launch_bwd_chain(D, H, Ul, Uu, stash, dy_flat, dh_dirs, dA, st);
    }
    if (e != hipSuccess) return hip_fail(e, "mdl_backward: reverse wavefront");
    if (dx_canvas) {
        Timed t("zero_fill");
        e = mdl::launch_zero_outside(D, dx_canvas, C, 1, st);
        if (e != hipSuccess) return hip_fail(e, "mdl_backward: zero fill");
    }
    if (ov_wg > 0) {
        // each wait at most ~2^15 clock cycles per dependent step of the layout (several times the reverse
        // wavefront's own time per step), at least 2^26 cycles
        const long long budget = ov_mode == 2 ? 0 : std::max<long long>(1ll << 26, (long long)L.max_depth << 15);
        {
            Timed t("wgrad_overlap");
            e = mdl::launch_wgrad2_claim(D, x_canvas, x_dtype, C, H, h_dirs, dA, Wx, part, want_dx ? dxp : nullptr,
                                         F, mdl::kClaimBeside, ov_wg, budget, 0, side->s);
        }
        if (e != hipSuccess) return hip_fail(e, "mdl_backward: weight gradients beside the reverse wavefront");
        if ((e = hipEventRecord(side->join, side->s)) != hipSuccess)
            return hip_fail(e, "mdl_backward: weight-gradient stream");
        {
            Timed t("wgrad");
            e = mdl::launch_wgrad2_claim(D, x_canvas, x_dtype, C, H, h_dirs, dA, Wx, part, want_dx ? dxp : nullptr,
                                         F, mdl::kClaimDrain, 0, 0, 0, st);
            if (e == hipSuccess && (e = hipStreamWaitEvent(st, side->join, 0)) == hipSuccess)
                e = mdl::launch_wgrad2_claim(D, x_canvas, x_dtype, C, H, h_dirs, dA, Wx, part,
                                             want_dx ? dxp : nullptr, F, mdl::kClaimAbandoned, 16, 0, 0, st);
            if (e == hipSuccess) e = mdl::launch_dx_sum(D, C, dxp, dx_flat, dx_canvas, st);
            if (e == hipSuccess) e = mdl::launch_wgrad_reduce(L.ngroups, C, H, part, dWx, dUl, dUu, db, st);
        }
        if (e != hipSuccess) return hip_fail(e, "mdl_backward: weight and input gradients");
    } else {
        Timed t("wgrad");
        e = mdl::launch_wgrad(D, x_canvas, x_dtype, C, H, h_dirs, dA, Wx, part, dxp, dWx, dUl, dUu, db, dx_flat,
                              dx_canvas, st);
        if (e != hipSuccess) return hip_fail(e, "mdl_backward: weight and input gradients");
    }
    if (lk) {
        // the memory-state projections' gradients, their partials in the partial-sum buffer the weight gradients
        // above are done with ([ngroups][4][2H][3H] fits in its [nparts][4][C+1+2H][5H])
        Timed t("wgrad_mem");
        e = mdl::launch_dv_leaky(D, H, stash, dA, part, dVl, dVu, st);
        if (e != hipSuccess) return hip_fail(e, "mdl_backward: memory-state projection gradients");
    }
    return MDL_OK;
    GUARD_END
}

static int check_conv(const char* fn, const mdl_layout* lk, const void* dk, const mdl_layout* lk1, const void* dk1,
                      int32_t H, int32_t kh, int32_t kw, int32_t Cout) {
    if (!lk || !dk || !lk1 || !dk1) return fail(MDL_EINVAL, std::string(fn) + ": null layout or descriptor");
    if (H < 1 || kh < 1 || kw < 1 || Cout < 1) return fail(MDL_EINVAL, std::string(fn) + ": non-positive size");
    const mdl::Layout& A = L_of(lk);
    const mdl::Layout& B = L_of(lk1);
    if (A.n != B.n) return fail(MDL_EINVAL, std::string(fn) + ": layouts hold different example counts");
    for (int e = 0; e < A.n; ++e) {
        const int h = A.real[4 * e + 2], w = A.real[4 * e + 3];
        if (B.real[4 * e + 2] != (h + kh - 1) / kh || B.real[4 * e + 3] != (w + kw - 1) / kw)
            return fail(MDL_EINVAL, std::string(fn) + ": level-(k+1) example sizes are not ceil(h/kh) x ceil(w/kw)");
    }
    return MDL_OK;
}

int mdl_blockconv_forward(const mdl_layout* lk, const void* d_desc_k, const mdl_layout* lk1, const void* d_desc_k1,
                          const float* h_dirs_k, int32_t H, int32_t kh, int32_t kw, const float* Wc, const float* bc,
                          int32_t Cout, float* x_canvas_k1, void* stream) {
    GUARD_BEGIN
    int rc = check_conv("mdl_blockconv_forward", lk, d_desc_k, lk1, d_desc_k1, H, kh, kw, Cout);
    if (rc) return rc;
    if (!h_dirs_k || !Wc || !bc || !x_canvas_k1) return fail(MDL_EINVAL, "mdl_blockconv_forward: null tensor");
    size_t lmax = 0;
    if ((rc = max_lds(lmax))) return rc;
    if (mdl::conv_fwd_lds(H, kh, kw, Cout) > lmax)
        return fail(MDL_EUNSUPPORTED, "mdl_blockconv_forward: weights and block tile exceed LDS");
    hipError_t e;
    {
        Timed t("conv_fwd");
        e = mdl::launch_conv_fwd(make_dev(lk, d_desc_k), make_dev(lk1, d_desc_k1), h_dirs_k, H, kh, kw, Wc, bc, Cout,
                                 x_canvas_k1, static_cast<hipStream_t>(stream));
    }
    if (e != hipSuccess) return hip_fail(e, "mdl_blockconv_forward");
    return MDL_OK;
    GUARD_END
}

int mdl_blockconv_workspace_size(const mdl_layout* lk1, int32_t H, int32_t kh, int32_t kw, int32_t Cout,
                                 size_t* bytes) {
    if (!lk1 || !bytes) return fail(MDL_EINVAL, "mdl_blockconv_workspace_size: null argument");
    if (H < 1 || kh < 1 || kw < 1 || Cout < 1) return fail(MDL_EINVAL, "mdl_blockconv_workspace_size: non-positive size");
    const mdl::Layout& B = L_of(lk1);
    mdl::Dev D{};
    D.N = B.real_pixels;
    D.Hc = B.Hc;
    D.Wc = B.Wc;
    const int64_t K = 4 * (int64_t)H * kh * kw;
    *bytes = sizeof(float) * (size_t)mdl::conv_nchunks(D) * (size_t)(Cout * (K + 1));
    return MDL_OK;
}

static int conv_bwd(const char* fn, const mdl_layout* lk, const void* d_desc_k, const mdl_layout* lk1,
                    const void* d_desc_k1, const float* h_dirs_k, int32_t H, int32_t kh, int32_t kw, const float* Wc,
                    int32_t Cout, const float* dx_canvas_k1, float* dh_dirs_k, float* dWc, float* dbc, void* ws,
                    size_t ws_bytes, bool fixed_scratch, void* stream) {
    int rc = check_conv(fn, lk, d_desc_k, lk1, d_desc_k1, H, kh, kw, Cout);
    if (rc) return rc;
    if (!h_dirs_k || !Wc || !dx_canvas_k1 || !dh_dirs_k || !dWc || !dbc || !ws)
        return fail(MDL_EINVAL, std::string(fn) + ": null tensor");
    const int64_t K = 4 * (int64_t)H * kh * kw;
    if (Cout * (K + 1) > 16 * 512) return fail(MDL_EUNSUPPORTED, std::string(fn) + ": Cout*(4*H*kh*kw+1) above 8192");
    size_t need = 0;
    mdl_blockconv_workspace_size(lk1, H, kh, kw, Cout, &need);
    if (ws_bytes < need) {
        if (fixed_scratch)
            return fail(MDL_ESIZE, std::string(fn) + ": the weight-gradient partials need " + std::to_string(need) +
                                       " bytes, above the library's fixed scratch of " + std::to_string(ws_bytes));
        return fail(MDL_ESIZE, std::string(fn) + ": workspace too small");
    }
    size_t lmax = 0;
    if ((rc = max_lds(lmax))) return rc;
    if (mdl::conv_wgrad_lds(H, kh, kw, Cout) > lmax || mdl::conv_data_lds(H, kh, kw, Cout) > lmax)
        return fail(MDL_EUNSUPPORTED, std::string(fn) + ": weight-gradient tile or weights exceed LDS");
    hipError_t e;
    {
        Timed t("conv_bwd");
        e = mdl::launch_conv_bwd(make_dev(lk, d_desc_k), make_dev(lk1, d_desc_k1), h_dirs_k, H, kh, kw, Wc, Cout,
                                 dx_canvas_k1, dh_dirs_k, dWc, dbc, static_cast<float*>(ws),
                                 static_cast<hipStream_t>(stream));
    }
    if (e != hipSuccess) return hip_fail(e, fn);
    return MDL_OK;
}

int mdl_blockconv_backward(const mdl_layout* lk, const void* d_desc_k, const mdl_layout* lk1, const void* d_desc_k1,
                           const float* h_dirs_k, int32_t H, int32_t kh, int32_t kw, const float* Wc, int32_t Cout,
                           const float* dx_canvas_k1, float* dh_dirs_k, float* dWc, float* dbc, void* ws,
                           size_t ws_bytes, void* stream) {
    GUARD_BEGIN
    return conv_bwd("mdl_blockconv_backward", lk, d_desc_k, lk1, d_desc_k1, h_dirs_k, H, kh, kw, Wc, Cout,
                    dx_canvas_k1, dh_dirs_k, dWc, dbc, ws, ws_bytes, false, stream);
    GUARD_END
}

int mdl_blockconv_backward_noalloc(const mdl_layout* lk, const void* d_desc_k, const mdl_layout* lk1,
                                   const void* d_desc_k1, const float* h_dirs_k, int32_t H, int32_t kh, int32_t kw,
                                   const float* Wc, int32_t Cout, const float* dx_canvas_k1, float* dh_dirs_k,
                                   float* dWc, float* dbc, void* stream) {
    GUARD_BEGIN
    const char* fn = "mdl_blockconv_backward_noalloc";
    int rc = check_conv(fn, lk, d_desc_k, lk1, d_desc_k1, H, kh, kw, Cout);
    if (rc) return rc;
    void* ws = nullptr;
    size_t cap = 0;
    const hipError_t e = mdl::conv_scratch(&ws, &cap);
    if (e != hipSuccess) return hip_fail(e, "mdl_blockconv_backward_noalloc: scratch address");
    return conv_bwd(fn, lk, d_desc_k, lk1, d_desc_k1, h_dirs_k, H, kh, kw, Wc, Cout, dx_canvas_k1, dh_dirs_k, dWc,
                    dbc, ws, cap, true, stream);
    GUARD_END
}

static int ctc_tmax(const mdl::Layout& L) {
    int t = 0;
    for (int e = 0; e < L.n; ++e) t = std::max(t, L.real[4 * e + 3]);
    return t;
}

static int check_ctc(const char* fn, const mdl_layout* layout, int32_t H, int32_t K, int32_t max_label) {
    if (!layout) return fail(MDL_EINVAL, std::string(fn) + ": null layout");
    if (H < 1 || K < 2 || max_label < 0)
        return fail(MDL_EINVAL, std::string(fn) + ": need H >= 1, K >= 2 and max_label >= 0");
    if (H > 1024 || K > 4096 || max_label > 65535)
        return fail(MDL_EUNSUPPORTED, std::string(fn) + ": H above 1024, K above 4096 or max_label above 65535");
    const int64_t T = ctc_tmax(L_of(layout));
    const int64_t S = 2 * (int64_t)max_label + 1;
    if (T * std::max<int64_t>(std::max<int64_t>(H, K), S) >= (int64_t(1) << 31))
        return fail(MDL_EOVERFLOW, std::string(fn) + ": frames times classes, hidden units or label states reach 2^31");
    return MDL_OK;
}

int mdl_ctc_workspace_size(const mdl_layout* layout, int32_t H, int32_t K, int32_t max_label, size_t* bytes) {
    GUARD_BEGIN
    if (!bytes) return fail(MDL_EINVAL, "mdl_ctc_workspace_size: null argument");
    int rc = check_ctc("mdl_ctc_workspace_size", layout, H, K, max_label);
    if (rc) return rc;
    const mdl::Layout& L = L_of(layout);
    *bytes = sizeof(float) * (size_t)mdl::ctc_ws(L.n, ctc_tmax(L), H, K, max_label).total;
    return MDL_OK;
    GUARD_END
}

int mdl_ctc_head(const mdl_layout* layout, const void* d_desc, const float* y_flat, int32_t H, const float* Wfc,
                 const float* bfc, int32_t K, const int32_t* labels, const int32_t* label_off, int64_t n_labels,
                 int32_t max_label, float* loss, float* dy_flat, float* dWfc, float* dbfc, void* ws,
                 size_t ws_bytes, void* stream) {
    GUARD_BEGIN
    int rc = check_ctc("mdl_ctc_head", layout, H, K, max_label);
    if (rc) return rc;
    if (!d_desc || !y_flat || !Wfc || !bfc || !label_off || !loss || !ws)
        return fail(MDL_EINVAL, "mdl_ctc_head: null tensor");
    if (n_labels < 0 || (n_labels > 0 && !labels)) return fail(MDL_EINVAL, "mdl_ctc_head: bad label array");
    if ((dWfc == nullptr) != (dbfc == nullptr))
        return fail(MDL_EINVAL, "mdl_ctc_head: give both dWfc and dbfc, or neither");
    const mdl::Layout& L = L_of(layout);
    const int Tmax = ctc_tmax(L);
    const size_t need = sizeof(float) * (size_t)mdl::ctc_ws(L.n, Tmax, H, K, max_label).total;
    if (ws_bytes < need) return fail(MDL_ESIZE, "mdl_ctc_head: workspace smaller than mdl_ctc_workspace_size");
    size_t lds = 0;
    rc = max_lds(lds);
    if (rc) return rc;
    hipError_t e;
    {
        Timed t("ctc_head");
        e = mdl::launch_ctc_head(make_dev(layout, d_desc), y_flat, H, Wfc, bfc, K, labels, label_off, n_labels,
                                 max_label, Tmax, static_cast<float*>(ws), loss, dy_flat, dWfc, dbfc, lds,
                                 static_cast<hipStream_t>(stream));
    }
    if (e != hipSuccess) return hip_fail(e, "mdl_ctc_head");
    return MDL_OK;
    GUARD_END
}

// Looks at another tile's word before a scan's tile forms what it waits for itself: about a millisecond, many times what
// a tile takes. None where mdl_set_scan_wait(0) leaves out the wait.
constexpr int kScanPolls = 1024;

// ---- the gated recurrence over packed sequences ---------------------------------------------------
static int check_dtype(const std::string& F, int32_t dtype) {
    if (dtype != MDL_F32 && dtype != MDL_BF16) return fail(MDL_EINVAL, F + ": unknown dtype");
    return MDL_OK;
}
// a row stride of at least `cols` elements whose largest element offset stays far inside 64 bits
static int check_stride(const std::string& F, const char* name, int64_t rows, int64_t cols, int64_t ld) {
    if (ld < cols) return fail(MDL_EINVAL, F + ": " + name + " below the row length");
    if (ld >= (int64_t(1) << 60) / std::max<int64_t>(rows, 1))
        return fail(MDL_EOVERFLOW, F + ": rows times " + name + " reach 2^60");
    return MDL_OK;
}
// as check_stride, for the kernels that keep strides in 32 bits
static int check_stride32(const std::string& F, const char* name, int64_t rows, int64_t cols, int64_t ld) {
    if (ld >= (int64_t(1) << 31)) return fail(MDL_EOVERFLOW, F + ": " + name + " reaches 2^31");
    return check_stride(F, name, rows, cols, ld);
}
// sizes and workspace of a scan; need receives the workspace bytes
static int check_scan(const std::string& F, int64_t T, int32_t D, int32_t dtype, size_t& need) {
    int rc = check_dtype(F, dtype);
    if (rc) return rc;
    if (T < 0 || D < 1) return fail(MDL_EINVAL, F + ": need T >= 0 and D >= 1");
    if (T >= (int64_t(1) << 60) / D) return fail(MDL_EOVERFLOW, F + ": rows times channels reach 2^60");
    const mdl::ScanPlan p = mdl::scan_plan(T, D, dtype);
    if (p.ntiles > mdl::kMaxLaunchThreads / 256 / p.ncb)
        return fail(MDL_EOVERFLOW, F + ": the launch exceeds 2^31 threads");
    need = p.total;
    return MDL_OK;
}
// the search for a tile's first sequence adds up to 63 to a count of them
static int check_sequences(const std::string& F, int32_t S) {
    if (S < 1) return fail(MDL_EINVAL, F + ": need S >= 1");
    if (S >= INT32_MAX - 63) return fail(MDL_EOVERFLOW, F + ": S reaches 2^31 - 64");
    return MDL_OK;
}
// Outputs that start where an input or another output does: tiles read their inputs again, and those of other tiles,
// after some have written. (Column blocks of one matrix lie between each other, so only the starts are compared.)
static int check_apart(const std::string& F, std::initializer_list<const void*> outs, std::initializer_list<const void*> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        if (!*o) continue;
        const bool over = std::count(ins.begin(), ins.end(), *o) || std::count(o + 1, outs.end(), *o);
        if (over) return fail(MDL_EINVAL, F + ": an output over an input or another output");
    }
    return MDL_OK;
}
// whether two arrays [S][D] of float share elements
static bool share_states(const void* a, const void* b, int32_t S, int32_t D) {
    if (!a || !b) return false;
    const uint64_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return (x > y ? x - y : y - x) / 4 < (uint64_t)S * (uint64_t)D;
}
static int check_ws(const std::string& F, const char* size_fn, size_t need, const void* ws, size_t ws_bytes) {
    if (need > 0 && !ws) return fail(MDL_EINVAL, F + ": null workspace");
    if (need > 0 && reinterpret_cast<uintptr_t>(ws) % 16) return fail(MDL_EINVAL, F + ": workspace not 16-byte aligned");
    if (ws_bytes < need) return fail(MDL_ESIZE, F + ": workspace smaller than " + size_fn);
    return MDL_OK;
}

int mdl_scan_workspace_size(int64_t T, int32_t D, int32_t dtype, size_t* bytes) {
    GUARD_BEGIN
    if (!bytes) return fail(MDL_EINVAL, "mdl_scan_workspace_size: null argument");
    size_t need = 0;
    const int rc = check_scan("mdl_scan_workspace_size", T, D, dtype, need);
    if (rc) return rc;
    *bytes = need;
    return MDL_OK;
    GUARD_END
}

int mdl_scan_forward(const int64_t* seq_off, int32_t S, int64_t T, int32_t D, int32_t dtype, int32_t reverse,
                     const void* zf, const void* g, const void* zo, int64_t ldz, const float* h0, void* y,
                     int64_t ldy, float* hT, void* ws, size_t ws_bytes, void* stream) {
    GUARD_BEGIN
    const std::string F("mdl_scan_forward");
    size_t need = 0;
    int rc = check_scan(F, T, D, dtype, need);
    if (rc) return rc;
    if ((rc = check_sequences(F, S))) return rc;
    if (!seq_off || (T > 0 && (!zf || !g || !y))) return fail(MDL_EINVAL, F + ": null tensor");
    if ((rc = check_stride32(F, "ldz", T, D, ldz)) || (rc = check_stride32(F, "ldy", T, D, ldy))) return rc;
    if ((rc = check_ws(F, "mdl_scan_workspace_size", need, ws, ws_bytes))) return rc;
    if (T > 0 && (rc = check_apart(F, {y, hT}, {zf, g, zo}))) return rc;
    if (share_states(h0, hT, S, D)) return fail(MDL_EINVAL, F + ": hT over h0");
    mdl::ScanArgs a{};
    a.off = seq_off;
    a.S = S;
    a.D = D;
    a.reverse = reverse != 0;
    a.polls = g_scan_wait.load() ? kScanPolls : -1;
    a.T = T;
    a.zf = zf;
    a.g = g;
    a.zo = zo;
    a.ldz = (int)ldz;
    a.ldy = (int)ldy;
    a.h0 = h0;
    a.y = y;
    a.hT = hT;
    hipError_t e;
    {
        Timed t("scan_fwd");
        e = mdl::launch_scan_fwd(a, dtype, ws, static_cast<hipStream_t>(stream));
    }
    if (e != hipSuccess) return hip_fail(e, F);
    return MDL_OK;
    GUARD_END
}

int mdl_scan_backward(const int64_t* seq_off, int32_t S, int64_t T, int32_t D, int32_t dtype, int32_t reverse,
                      const void* zf, const void* g, const void* zo, int64_t ldz, const float* h0, const void* dy,
                      int64_t ldy, const float* dhT, void* dzf, void* dg, void* dzo, int64_t ldd, float* dh0,
                      void* ws, size_t ws_bytes, void* stream) {
    GUARD_BEGIN
    const std::string F("mdl_scan_backward");
    size_t need = 0;
    int rc = check_scan(F, T, D, dtype, need);
    if (rc) return rc;
    if ((rc = check_sequences(F, S))) return rc;
    if (!seq_off || (T > 0 && (!zf || !g || !dy || !dzf || !dg))) return fail(MDL_EINVAL, F + ": null tensor");
    if (T > 0 && (zo == nullptr) != (dzo == nullptr)) return fail(MDL_EINVAL, F + ": dzo goes with zo, and only with it");
    if ((rc = check_stride32(F, "ldz", T, D, ldz)) || (rc = check_stride32(F, "ldy", T, D, ldy)) ||
        (rc = check_stride32(F, "ldd", T, D, ldd)))
        return rc;
    if ((rc = check_ws(F, "mdl_scan_workspace_size", need, ws, ws_bytes))) return rc;
    if (T > 0 && (rc = check_apart(F, {dzf, dg, dzo}, {zf, g, zo, dy}))) return rc;
    if (share_states(h0, dh0, S, D) || share_states(dhT, dh0, S, D))
        return fail(MDL_EINVAL, F + ": dh0 over h0 or dhT");
    mdl::ScanArgs a{};
    a.off = seq_off;
    a.S = S;
    a.D = D;
    a.reverse = reverse != 0;
    a.polls = g_scan_wait.load() ? kScanPolls : -1;
    a.T = T;
    a.zf = zf;
    a.g = g;
    a.zo = zo;
    a.dy = dy;
    a.ldz = (int)ldz;
    a.ldy = (int)ldy;
    a.ldd = (int)ldd;
    a.h0 = h0;
    a.dhT = dhT;
    a.dzf = dzf;
    a.dg = dg;
    a.dzo = dzo;
    a.dh0 = dh0;
    hipError_t e;
    {
        Timed t("scan_bwd");
        e = mdl::launch_scan_bwd(a, dtype, ws, static_cast<hipStream_t>(stream));
    }
    if (e != hipSuccess) return hip_fail(e, F);
    return MDL_OK;
    GUARD_END
}

int mdl_scan_step(int32_t S, int32_t D, int32_t dtype, const void* zf, const void* g, const void* zo, int64_t ldz,
                  const int32_t* slots, int32_t n_slots, const float* h_in, float* h_out, void* y, int64_t ldy,
                  void* stream) {
    GUARD_BEGIN
    const std::string F("mdl_scan_step");
    int rc = check_dtype(F, dtype);
    if (rc) return rc;
    if (S < 1 || D < 1 || n_slots < 1) return fail(MDL_EINVAL, F + ": need S, D and n_slots >= 1");
    if (!zf || !g || !h_in || !h_out || !y) return fail(MDL_EINVAL, F + ": null tensor");
    if ((int64_t)S * D > mdl::kMaxLaunchThreads) return fail(MDL_EOVERFLOW, F + ": S times D exceeds 2^31");
    if (!slots && n_slots < S) return fail(MDL_EINVAL, F + ": n_slots below S without slots");
    if ((rc = check_stride(F, "ldz", S, D, ldz)) || (rc = check_stride(F, "ldy", S, D, ldy))) return rc;
    hipError_t e;
    {
        Timed t("scan_step");
        e = mdl::launch_scan_step(S, D, dtype, zf, g, zo, ldz, slots, n_slots, h_in, h_out, y, ldy,
                                  static_cast<hipStream_t>(stream));
    }
    if (e != hipSuccess) return hip_fail(e, F);
    return MDL_OK;
    GUARD_END
}

// ---- the norms before and after a block --------------------------------------------------------------
static int check_norm(const std::string& F, int64_t N, int32_t D, int32_t dtype) {
    int rc = check_dtype(F, dtype);
    if (rc) return rc;
    if (N < 0 || D < 1) return fail(MDL_EINVAL, F + ": need N >= 0 and D >= 1");
    if (D > mdl::norm_max_d()) return fail(MDL_EUNSUPPORTED, F + ": D above " + std::to_string(mdl::norm_max_d()));
    if (N >= (int64_t(1) << 40)) return fail(MDL_EOVERFLOW, F + ": N reaches 2^40");
    return MDL_OK;
}
static int check_norm_parts(const std::string& F, const mdl::NormArgs& a) {
    if (a.N > 0 && !a.x) return fail(MDL_EINVAL, F + ": null tensor");
    if (a.N > 0 && !a.z && (a.u || a.w_post || a.scale))
        return fail(MDL_EINVAL, F + ": a gate, w_post or scale without z");
    if (!(a.eps >= 0.f && a.eps < INFINITY)) return fail(MDL_EINVAL, F + ": eps must be finite and >= 0");
    int rc = check_stride(F, "ldx", a.N, a.D, a.ldx);
    if (!rc && a.z) rc = check_stride(F, "ldz", a.N, a.D, a.ldz);
    if (!rc && a.u) rc = check_stride(F, "ldu", a.N, a.D, a.ldu);
    if (!rc) rc = check_stride(F, "ldr", a.N, a.D, a.ldr);
    return rc;
}

int mdl_blocknorm_forward(int64_t N, int32_t D, int32_t dtype, const void* x, int64_t ldx, const void* z, int64_t ldz,
                          const void* u, int64_t ldu, const float* w_post, const float* scale, const float* w_pre,
                          float eps, void* r, void* v, int64_t ldr, void* stream) {
    GUARD_BEGIN
    const std::string F("mdl_blocknorm_forward");
    int rc = check_norm(F, N, D, dtype);
    if (rc) return rc;
    mdl::NormArgs a{};
    a.N = N;
    a.D = D;
    a.x = x;
    a.z = z;
    a.u = u;
    a.ldx = ldx;
    a.ldz = ldz;
    a.ldu = ldu;
    a.ldr = ldr;
    a.w_post = w_post;
    a.scale = scale;
    a.w_pre = w_pre;
    a.eps = eps;
    a.inv_d = 1.f / (float)D;
    a.r = r;
    a.v = v;
    if ((rc = check_norm_parts(F, a))) return rc;
    if (N > 0) {
        if ((z == nullptr) != (r == nullptr)) return fail(MDL_EINVAL, F + ": r goes with z, and only with it");
        if ((w_pre == nullptr) != (v == nullptr)) return fail(MDL_EINVAL, F + ": v goes with w_pre, and only with it");
        if (!r && !v) return fail(MDL_EINVAL, F + ": nothing to compute");
    }
    hipError_t e;
    {
        Timed t("norm_fwd");
        e = mdl::launch_norm_fwd(a, dtype, static_cast<hipStream_t>(stream));
    }
    if (e != hipSuccess) return hip_fail(e, F);
    return MDL_OK;
    GUARD_END
}

int mdl_blocknorm_workspace_size(int64_t N, int32_t D, int32_t dtype, size_t* bytes) {
    GUARD_BEGIN
    if (!bytes) return fail(MDL_EINVAL, "mdl_blocknorm_workspace_size: null argument");
    const int rc = check_norm("mdl_blocknorm_workspace_size", N, D, dtype);
    if (rc) return rc;
    *bytes = mdl::norm_bwd_ws(N, D, dtype);
    return MDL_OK;
    GUARD_END
}

int mdl_blocknorm_backward(int64_t N, int32_t D, int32_t dtype, const void* x, int64_t ldx, const void* z, int64_t ldz,
                           const void* u, int64_t ldu, const float* w_post, const float* scale, const float* w_pre,
                           float eps, const void* dr, const void* dv, int64_t ldr, void* dx, void* dz, void* du,
                           int64_t ldd, float* dw_post, float* dscale, float* dw_pre, void* ws, size_t ws_bytes,
                           void* stream) {
    GUARD_BEGIN
    const std::string F("mdl_blocknorm_backward");
    int rc = check_norm(F, N, D, dtype);
    if (rc) return rc;
    mdl::NormArgs a{};
    a.N = N;
    a.D = D;
    a.x = x;
    a.z = z;
    a.u = u;
    a.ldx = ldx;
    a.ldz = ldz;
    a.ldu = ldu;
    a.ldr = ldr;
    a.ldd = ldd;
    a.w_post = w_post;
    a.scale = scale;
    a.w_pre = w_pre;
    a.eps = eps;
    a.inv_d = 1.f / (float)D;
    a.dr = dr;
    a.dv = dv;
    a.dx = dx;
    a.dz = dz;
    a.du = du;
    a.part = static_cast<float*>(ws);
    if ((rc = check_norm_parts(F, a))) return rc;
    if ((rc = check_stride(F, "ldd", N, D, ldd))) return rc;
    if (N > 0) {
        if (!dx) return fail(MDL_EINVAL, F + ": null tensor");
        if ((z == nullptr) != (dz == nullptr) || (u == nullptr) != (du == nullptr))
            return fail(MDL_EINVAL, F + ": dz goes with z and du with u, and only with them");
        if ((w_pre == nullptr) != (dv == nullptr)) return fail(MDL_EINVAL, F + ": dv goes with w_pre, and only with it");
        if (!dr && !dv) return fail(MDL_EINVAL, F + ": neither dr nor dv");
    }
    if ((w_post == nullptr) != (dw_post == nullptr) || (scale == nullptr) != (dscale == nullptr) ||
        (w_pre == nullptr) != (dw_pre == nullptr))
        return fail(MDL_EINVAL, F + ": each weight's gradient goes with the weight, and only with it");
    if ((rc = check_ws(F, "mdl_blocknorm_workspace_size", mdl::norm_bwd_ws(N, D, dtype), ws, ws_bytes))) return rc;
    hipError_t e;
    {
        Timed t("norm_bwd");
        e = mdl::launch_norm_bwd(a, dtype, dw_post, dscale, dw_pre, static_cast<hipStream_t>(stream));
    }
    if (e != hipSuccess) return hip_fail(e, F);
    return MDL_OK;
    GUARD_END
}

// ---- distillation from a teacher's top logits ----------------------------------------------------------
int mdl_distill(int64_t N, int32_t V, int32_t k, int32_t dtype, const void* z, int64_t ldz, const int32_t* ids,
                const void* t, int32_t t_dtype, const float* w, float tau, float* loss, void* dz, int64_t ldd,
                void* stream) {
    GUARD_BEGIN
    const std::string F("mdl_distill");
    int rc = check_dtype(F, dtype);
    if (rc || (rc = check_dtype(F, t_dtype))) return rc;
    if (N < 0 || V < 1 || k < 1 || k > V) return fail(MDL_EINVAL, F + ": need N >= 0, V >= 1 and k in [1, V]");
    if (k > mdl::distill_max_k()) return fail(MDL_EUNSUPPORTED, F + ": k above " + std::to_string(mdl::distill_max_k()));
    if (N >= (int64_t(1) << 40)) return fail(MDL_EOVERFLOW, F + ": N reaches 2^40");
    if (N > 0 && (!z || !ids || !t || !loss)) return fail(MDL_EINVAL, F + ": null tensor");
    if (!(tau >= 1e-30f && tau < INFINITY)) return fail(MDL_EINVAL, F + ": tau must be finite and at least 1e-30");
    if ((rc = check_stride(F, "ldz", N, V, ldz))) return rc;
    if (dz && (rc = check_stride(F, "ldd", N, V, ldd))) return rc;
    hipError_t e;
    {
        Timed tm("distill");
        e = mdl::launch_distill(N, V, k, dtype, z, ldz, ids, t, t_dtype, w, tau, loss, dz, ldd,
                                static_cast<hipStream_t>(stream));
    }
    if (e != hipSuccess) return hip_fail(e, F);
    return MDL_OK;
    GUARD_END
}

// ---- linear attention with a decay for each head -------------------------------------------------------
// a head's sizes, as all attention calls take them
static int check_heads(const std::string& F, int32_t H, int32_t Dk, int32_t Dv, int32_t dtype) {
    int rc = check_dtype(F, dtype);
    if (rc) return rc;
    if (H < 1 || Dk < 1 || Dv < 1) return fail(MDL_EINVAL, F + ": need H, Dk, Dv >= 1");
    if (Dk > mdl::linattn_max_d() || Dv > mdl::linattn_max_d())
        return fail(MDL_EUNSUPPORTED, F + ": Dk or Dv above " + std::to_string(mdl::linattn_max_d()));
    if (H > 65535) return fail(MDL_EUNSUPPORTED, F + ": H above 65535");
    return MDL_OK;
}
// sizes of a call over sequences; need receives the workspace bytes
static int check_attn(const std::string& F, int32_t S, int64_t T, int32_t H, int32_t Dk, int32_t Dv, int32_t dtype,
                      size_t& need) {
    int rc = check_heads(F, H, Dk, Dv, dtype);
    if (rc || (rc = check_sequences(F, S))) return rc;
    if (T < 0) return fail(MDL_EINVAL, F + ": need T >= 0");
    if (T >= (int64_t(1) << 36)) return fail(MDL_EOVERFLOW, F + ": T reaches 2^36");
    const mdl::AttnPlan p = mdl::attn_plan(S, T, H, Dk, Dv);
    const int64_t most = mdl::kMaxLaunchThreads / 512;
    if (S > most / p.chain_blocks || T / p.L + S > most / H) return fail(MDL_EOVERFLOW, F + ": the launch exceeds 2^31 threads");
    need = p.total;
    return MDL_OK;
}
// as check_stride, for the kernels whose blocks of rows keep their offsets in 31 bits
static int check_stride23(const std::string& F, const char* name, int64_t rows, int64_t cols, int64_t ld) {
    if (ld >= (int64_t(1) << 23)) return fail(MDL_EOVERFLOW, F + ": " + name + " reaches 2^23");
    return check_stride(F, name, rows, cols, ld);
}
// whether `bytes` bytes at a and b share any
static bool share_bytes(const void* a, const void* b, uint64_t bytes) {
    if (!a || !b) return false;
    const uint64_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return (x > y ? x - y : y - x) < bytes;
}
static uint64_t state_bytes(int32_t S, int32_t H, int32_t Dk, int32_t Dv) {
    return (uint64_t)S * (uint64_t)H * (uint64_t)Dk * (uint64_t)Dv * 4;
}

int mdl_linattn_workspace_size(int32_t S, int64_t T, int32_t H, int32_t Dk, int32_t Dv, int32_t dtype, size_t* bytes) {
    GUARD_BEGIN
    if (!bytes) return fail(MDL_EINVAL, "mdl_linattn_workspace_size: null argument");
    size_t need = 0;
    const int rc = check_attn("mdl_linattn_workspace_size", S, T, H, Dk, Dv, dtype, need);
    if (rc) return rc;
    *bytes = need;
    return MDL_OK;
    GUARD_END
}

int mdl_linattn_forward(const int64_t* seq_off, int32_t S, int64_t T, int32_t H, int32_t Dk, int32_t Dv, int32_t dtype,
                        int32_t reverse, const float* decay, float scale, const void* q, int64_t ldq, const void* k,
                        int64_t ldk, const void* v, int64_t ldv, const float* h0, void* y, int64_t ldy, float* hT,
                        void* ws, size_t ws_bytes, void* stream) {
    GUARD_BEGIN
    const std::string F("mdl_linattn_forward");
    size_t need = 0;
    int rc = check_attn(F, S, T, H, Dk, Dv, dtype, need);
    if (rc) return rc;
    if (!seq_off || !decay || (T > 0 && (!q || !k || !v || !y))) return fail(MDL_EINVAL, F + ": null tensor");
    const int64_t nk = (int64_t)H * Dk, nv = (int64_t)H * Dv;
    if ((rc = check_stride23(F, "ldq", T, nk, ldq)) || (rc = check_stride23(F, "ldk", T, nk, ldk)) ||
        (rc = check_stride23(F, "ldv", T, nv, ldv)) || (rc = check_stride23(F, "ldy", T, nv, ldy)))
        return rc;
    if ((rc = check_ws(F, "mdl_linattn_workspace_size", need, ws, ws_bytes))) return rc;
    if ((rc = check_apart(F, {hT}, {seq_off, decay}))) return rc;
    if (T > 0 && (rc = check_apart(F, {y, hT}, {seq_off, decay, q, k, v, h0}))) return rc;
    if (share_bytes(h0, hT, state_bytes(S, H, Dk, Dv))) return fail(MDL_EINVAL, F + ": hT over h0");
    mdl::AttnArgs a{};
    a.off = seq_off;
    a.S = S;
    a.H = H;
    a.Dk = Dk;
    a.Dv = Dv;
    a.reverse = reverse != 0;
    a.T = T;
    a.decay = decay;
    a.scale = scale;
    a.q = q;
    a.k = k;
    a.v = v;
    a.ldq = ldq;
    a.ldk = ldk;
    a.ldv = ldv;
    a.h0 = h0;
    a.y = y;
    a.ldy = ldy;
    a.hT = hT;
    hipError_t e;
    {
        Timed t("attn_fwd");
        e = mdl::launch_attn_fwd(a, dtype, ws, static_cast<hipStream_t>(stream));
    }
    if (e != hipSuccess) return hip_fail(e, F);
    return MDL_OK;
    GUARD_END
}

int mdl_linattn_backward(const int64_t* seq_off, int32_t S, int64_t T, int32_t H, int32_t Dk, int32_t Dv, int32_t dtype,
                         int32_t reverse, const float* decay, float scale, const void* q, int64_t ldq, const void* k,
                         int64_t ldk, const void* v, int64_t ldv, const float* h0, const void* dy, int64_t lddy,
                         const float* dhT, void* dq, int64_t lddq, void* dk, int64_t lddk, void* dv, int64_t lddv,
                         float* dh0, void* ws, size_t ws_bytes, void* stream) {
    GUARD_BEGIN
    const std::string F("mdl_linattn_backward");
    size_t need = 0;
    int rc = check_attn(F, S, T, H, Dk, Dv, dtype, need);
    if (rc) return rc;
    if (!seq_off || !decay || (T > 0 && (!q || !k || !v || !dy || !dq || !dk || !dv)))
        return fail(MDL_EINVAL, F + ": null tensor");
    const int64_t nk = (int64_t)H * Dk, nv = (int64_t)H * Dv;
    if ((rc = check_stride23(F, "ldq", T, nk, ldq)) || (rc = check_stride23(F, "ldk", T, nk, ldk)) ||
        (rc = check_stride23(F, "ldv", T, nv, ldv)) || (rc = check_stride23(F, "lddy", T, nv, lddy)) ||
        (rc = check_stride23(F, "lddq", T, nk, lddq)) || (rc = check_stride23(F, "lddk", T, nk, lddk)) ||
        (rc = check_stride23(F, "lddv", T, nv, lddv)))
        return rc;
    if ((rc = check_ws(F, "mdl_linattn_workspace_size", need, ws, ws_bytes))) return rc;
    if ((rc = check_apart(F, {dh0}, {seq_off, decay}))) return rc;
    if (T > 0 && (rc = check_apart(F, {dq, dk, dv, dh0}, {seq_off, decay, q, k, v, dy, h0, dhT}))) return rc;
    if (share_bytes(h0, dh0, state_bytes(S, H, Dk, Dv)) || share_bytes(dhT, dh0, state_bytes(S, H, Dk, Dv)))
        return fail(MDL_EINVAL, F + ": dh0 over h0 or dhT");
    mdl::AttnArgs a{};
    a.off = seq_off;
    a.S = S;
    a.H = H;
    a.Dk = Dk;
    a.Dv = Dv;
    a.reverse = reverse != 0;
    a.T = T;
    a.decay = decay;
    a.scale = scale;
    a.q = q;
    a.k = k;
    a.v = v;
    a.dy = dy;
    a.ldq = ldq;
    a.ldk = ldk;
    a.ldv = ldv;
    a.lddy = lddy;
    a.h0 = h0;
    a.dhT = dhT;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.lddq = lddq;
    a.lddk = lddk;
    a.lddv = lddv;
    a.dh0 = dh0;
    hipError_t e;
    {
        Timed t("attn_bwd");
        e = mdl::launch_attn_bwd(a, dtype, ws, static_cast<hipStream_t>(stream));
    }
    if (e != hipSuccess) return hip_fail(e, F);
    return MDL_OK;
    GUARD_END
}

int mdl_linattn_step(int32_t S, int32_t H, int32_t Dk, int32_t Dv, int32_t dtype, const float* decay, float scale,
                     const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                     const int32_t* slots, int32_t n_slots, const float* h_in, float* h_out, void* y, int64_t ldy,
                     void* stream) {
    GUARD_BEGIN
    const std::string F("mdl_linattn_step");
    int rc = check_heads(F, H, Dk, Dv, dtype);
    if (rc) return rc;
    if (S < 1 || n_slots < 1) return fail(MDL_EINVAL, F + ": need S and n_slots >= 1");
    if (!decay || !q || !k || !v || !h_in || !h_out || !y) return fail(MDL_EINVAL, F + ": null tensor");
    if ((int64_t)S * H > mdl::kMaxLaunchThreads / 256) return fail(MDL_EOVERFLOW, F + ": the launch exceeds 2^31 threads");
    if (!slots && n_slots < S) return fail(MDL_EINVAL, F + ": n_slots below S without slots");
    const int64_t nk = (int64_t)H * Dk, nv = (int64_t)H * Dv;
    if ((rc = check_stride(F, "ldq", S, nk, ldq)) || (rc = check_stride(F, "ldk", S, nk, ldk)) ||
        (rc = check_stride(F, "ldv", S, nv, ldv)) || (rc = check_stride(F, "ldy", S, nv, ldy)))
        return rc;
    if ((rc = check_apart(F, {y, h_out}, {q, k, v, decay, slots})) || (rc = check_apart(F, {y}, {h_in}))) return rc;
    // a row's states are read and written by one workgroup only where both arrays are one
    if (h_in != h_out && share_bytes(h_in, h_out, state_bytes(n_slots, H, Dk, Dv)))
        return fail(MDL_EINVAL, F + ": h_out over a part of h_in");
    mdl::AttnArgs a{};
    a.S = S;
    a.H = H;
    a.Dk = Dk;
    a.Dv = Dv;
    a.decay = decay;
    a.scale = scale;
    a.q = q;
    a.k = k;
    a.v = v;
    a.ldq = ldq;
    a.ldk = ldk;
    a.ldv = ldv;
    a.y = y;
    a.ldy = ldy;
    hipError_t e;
    {
        Timed t("attn_step");
        e = mdl::launch_attn_step(a, dtype, slots, n_slots, h_in, h_out, static_cast<hipStream_t>(stream));
    }
    if (e != hipSuccess) return hip_fail(e, F);
    return MDL_OK;
    GUARD_END
}

// ---- dropout ---------------------------------------------------------------------------------------------
int mdl_dropout(int64_t N, int32_t D, int32_t dtype, const void* x, int64_t ldx, const void* r, int64_t ldr, float p,
                const uint64_t* rng, void* y, int64_t ldy, void* stream) {
    GUARD_BEGIN
    const std::string F("mdl_dropout");
    int rc = check_dtype(F, dtype);
    if (rc) return rc;
    if (N < 0 || D < 1) return fail(MDL_EINVAL, F + ": need N >= 0 and D >= 1");
    if (!(p >= 0.f && p < 1.f)) return fail(MDL_EINVAL, F + ": p must lie in [0, 1)");
    const int cut = (int)std::lrint((double)p * 65536.0);
    if (cut > 65535) return fail(MDL_EINVAL, F + ": p rounds to 1 in steps of 2^-16");
    if (!rng || (N > 0 && (!x || !y))) return fail(MDL_EINVAL, F + ": null tensor");
    if (reinterpret_cast<uintptr_t>(rng) % 8) return fail(MDL_EINVAL, F + ": rng not 8-byte aligned");
    if ((rc = check_stride(F, "ldx", N, D, ldx)) || (rc = check_stride(F, "ldy", N, D, ldy))) return rc;
    if (r && (rc = check_stride(F, "ldr", N, D, ldr))) return rc;
    if ((rc = check_apart(F, {y}, {rng}))) return rc;
    // elements are read and written by the same thread only where both lie alike
    if (N > 1 && ((y == x && ldy != ldx) || (y == r && ldy != ldr)))
        return fail(MDL_EINVAL, F + ": y over x or r at another stride");
    if (N > mdl::dropout_max_groups() / (((int64_t)D + 7) / 8))
        return fail(MDL_EOVERFLOW, F + ": the launch exceeds 2^31 threads");
    hipError_t e;
    {
        Timed t("dropout");
        e = mdl::launch_dropout(N, D, dtype, x, ldx, r, ldr, cut, rng, y, ldy, static_cast<hipStream_t>(stream));
    }
    if (e != hipSuccess) return hip_fail(e, F);
    return MDL_OK;
    GUARD_END
}

// ---- cross entropy over a vocabulary ---------------------------------------------------------------------
static int check_vocab(const std::string& F, int64_t N, int32_t D, int32_t V, int32_t dtype, bool grads, size_t& need) {
    int rc = check_dtype(F, dtype);
    if (rc) return rc;
    if (N < 0 || D < 1 || V < 1) return fail(MDL_EINVAL, F + ": need N >= 0, D >= 1 and V >= 1");
    if (D > mdl::vocab_max_d()) return fail(MDL_EUNSUPPORTED, F + ": D above " + std::to_string(mdl::vocab_max_d()));
    if (V > mdl::vocab_max_classes())
        return fail(MDL_EUNSUPPORTED, F + ": V above " + std::to_string(mdl::vocab_max_classes()));
    // the widest launches: 256 threads for each 256 values of dh or dW, and for each tile of the logits
    const int64_t most = mdl::kMaxLaunchThreads, cols = ((int64_t)D + 255) / 256 * 256;
    if (N > most / cols || N > most / (((int64_t)V + 127) / 128) || V > most / cols)
        return fail(MDL_EOVERFLOW, F + ": a launch exceeds 2^31 threads");
    need = mdl::vocab_plan(N, D, V, dtype, grads).total;
    return MDL_OK;
}

int mdl_vocab_loss_workspace_size(int64_t N, int32_t D, int32_t V, int32_t dtype, int32_t grads, size_t* bytes) {
    GUARD_BEGIN
    if (!bytes) return fail(MDL_EINVAL, "mdl_vocab_loss_workspace_size: null argument");
    size_t need = 0;
    const int rc = check_vocab("mdl_vocab_loss_workspace_size", N, D, V, dtype, grads != 0, need);
    if (rc) return rc;
    *bytes = need;
    return MDL_OK;
    GUARD_END
}

int mdl_vocab_loss(int64_t N, int32_t D, int32_t V, int32_t dtype, const void* h, int64_t ldh, const void* W,
                   const int32_t* ids, const float* w, float* loss, void* dh, int64_t lddh, void* dW, void* ws,
                   size_t ws_bytes, void* stream) {
    GUARD_BEGIN
    const std::string F("mdl_vocab_loss");
    size_t need = 0;
    int rc = check_vocab(F, N, D, V, dtype, dW != nullptr, need);
    if (rc) return rc;
    if (!W || (N > 0 && (!h || !ids || !loss))) return fail(MDL_EINVAL, F + ": null tensor");
    if (N > 0 && (dh == nullptr) != (dW == nullptr)) return fail(MDL_EINVAL, F + ": dh and dW go together");
    if ((rc = check_stride(F, "ldh", N, D, ldh))) return rc;
    if (dh && (rc = check_stride(F, "lddh", N, D, lddh))) return rc;
    if (D % (dtype == MDL_BF16 ? 8 : 4) == 0 && reinterpret_cast<uintptr_t>(W) % 16)
        return fail(MDL_EINVAL, F + ": W not 16-byte aligned");
    if ((rc = check_ws(F, "mdl_vocab_loss_workspace_size", need, ws, ws_bytes))) return rc;
    if ((rc = check_apart(F, {dW, loss}, {h, W, ids, w, dh})) || (rc = check_apart(F, {dh}, {W, ids, w}))) return rc;
    const mdl::VocabArgs a{N, D, V, h, W, ldh, lddh, ids, w, loss, dh, dW};
    hipError_t e;
    {
        Timed t("vocab_loss");
        e = mdl::launch_vocab(a, dtype, ws, static_cast<hipStream_t>(stream));
    }
    if (e != hipSuccess) return hip_fail(e, F);
    return MDL_OK;
    GUARD_END
}

int mdl_set_scan_wait(int32_t on) {
    if (on < 0 || on > 1) return fail(MDL_EINVAL, "mdl_set_scan_wait: on must be 0 or 1");
    g_scan_wait.store(on != 0);
    return MDL_OK;
}

int mdl_set_wgrad_overlap(int32_t mode) {
    if (mode < 0 || mode > 2) return fail(MDL_EINVAL, "mdl_set_wgrad_overlap: mode must be 0, 1 or 2");
    g_overlap.store(mode);
    return MDL_OK;
}

int mdl_timing(int32_t enable) {
    std::lock_guard<std::mutex> lk(g_tmu);
    g_timing = enable != 0;
    return MDL_OK;
}

int mdl_timing_only(const char* group) {
    if (group && std::strlen(group) >= 32) return fail(MDL_EINVAL, "mdl_timing_only: group name too long");
    std::lock_guard<std::mutex> lk(g_tmu);
    g_timing_only = group ? group : "";
    return MDL_OK;
}

int mdl_timing_report(int32_t max, char* names, double* total_ms, int64_t* launches, int32_t* count) {
    GUARD_BEGIN
    if (max < 0 || !count || (max > 0 && (!names || !total_ms || !launches)))
        return fail(MDL_EINVAL, "mdl_timing_report: bad arguments");
    std::lock_guard<std::mutex> lk(g_tmu);
    std::map<std::string, std::pair<double, int64_t>> acc;
    std::vector<std::string> order;
    int rc = MDL_OK;
    for (auto& t : g_tlog) {
        float ms = 0.f;
        hipError_t e = hipEventSynchronize(t.ev.back());
        if (e == hipSuccess) e = hipEventElapsedTime(&ms, t.ev.front(), t.ev.back());
        if (e != hipSuccess && rc == MDL_OK) rc = hip_fail(e, "mdl_timing_report");
        if (!acc.count(t.name)) order.push_back(t.name);
        acc[t.name].first += ms;
        acc[t.name].second += 1;
        for (hipEvent_t ev : t.ev) g_event_pool.push_back(ev);
    }
    g_tlog.clear();
    int k = 0;
    for (const auto& nm : order) {
        if (k >= max) break;
        std::memset(names + 32 * k, 0, 32);
        std::strncpy(names + 32 * k, nm.c_str(), 31);
        total_ms[k] = acc[nm].first;
        launches[k] = acc[nm].second;
        ++k;
    }
    *count = k;
    return rc;
    GUARD_END
}

const char* mdl_last_error(void) { return g_err.c_str(); }

}  // extern "C"
