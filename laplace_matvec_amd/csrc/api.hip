// C ABI of the LAPLEX library: plans, argument checks, dispatch, timing.
//
// The operator and its fast algorithm follow the technical summary of
// "LAPLEX: The FFT of Learnable Laplace Kernels" (§2.1 operator, §2.2 scan
// algebra, general case and Gram); see include/laplex.h for the contract.
//
// Every argument check runs before the first HIP call, so invalid calls are
// rejected on any host, GPU or not.  Device memory comes from the library's
// caching allocator below (freed blocks kept per device and handed out
// again, each ordered after its last use by an event), so repeated plans and
// growing workspaces do not pay for fresh allocations.
#include <hip/hip_runtime.h>

#include <cstdlib>
#include <cfloat>
#include <cmath>
#include <cstring>
#include <mutex>
#include <string>
#include <vector>

#include "laplex.h"
#include "lx_internal.h"

namespace {

thread_local std::string g_last_error;

// Longest anchor side.  Permutations are uint32, and the backward replay
// forms its gather offsets as 32-bit byte offsets from a uniform base, so
// every element index times 4 must fit in 32 bits: n <= 2^30.
constexpr int64_t kMaxLen = (int64_t)1 << 30;

laplex_status fail(laplex_status st, const std::string& msg)
{
    g_last_error = msg;
    return st;
}

// Messages without formatting: nothing to throw at the C entry.
laplex_status fail(laplex_status st, const char* msg) noexcept
{
    try {
        g_last_error = msg;
    } catch (...) {
        g_last_error.clear();
    }
    return st;
}

laplex_status from_hip(hipError_t e, const char* where) noexcept
{
    if (e == hipSuccess) return LAPLEX_OK;
    laplex_status st = LAPLEX_ERR_DEVICE;
    if (e == hipErrorOutOfMemory || e == hipErrorMemoryAllocation) st = LAPLEX_ERR_OUT_OF_MEMORY;
    if (e == hipErrorNoDevice || e == hipErrorInvalidDevice) st = LAPLEX_ERR_NO_DEVICE;
    try {
        return fail(st, std::string(where) + ": " + hipGetErrorString(e));
    } catch (...) {
        return st;
    }
}

#define LX_TRY(call, where)                                          \
    do {                                                             \
        const laplex_status lx_s_ = from_hip((call), (where));       \
        if (lx_s_ != LAPLEX_OK) return lx_s_;                        \
    } while (0)

inline int64_t pad64(int64_t x) { return (x + 63) & ~(int64_t)63; }
inline size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }

// ------------------------------------------------------- caching allocator
//
// Device memory for plans, workspaces and sort scratch.  A layer whose
// anchors change every training step makes and drops a plan per step, tens
// of GB each time at n = 2^30, so freed blocks are kept per device and
// handed out again (best fit, at most twice the request) instead of going
// back to the driver.  A block freed on stream s carries an event recorded
// on s at the free; whoever takes it next orders its stream after that
// event, so reuse across streams is safe.  When the driver is out of
// memory, the cached blocks are released and the allocation is retried.
// One event recorded at a free, shared by the blocks freed together.
struct FreeEvent {
    hipEvent_t ev;
    int refs;
};
struct CachedBlock {
    void* ptr;
    size_t bytes;
    FreeEvent* freed;  // recorded at the free (null: idle already)
};
struct DeviceCache {
    std::mutex mu;
    std::vector<CachedBlock> idle;
    std::vector<std::pair<void*, size_t>> live;
    std::vector<hipEvent_t> events;
};
std::mutex g_cache_mu;
std::vector<DeviceCache*> g_caches;

DeviceCache& cache_for(int dev)
{
    std::lock_guard<std::mutex> lk(g_cache_mu);
    while ((int)g_caches.size() <= dev) g_caches.push_back(new DeviceCache());
    return *g_caches[dev];
}

size_t round_block(size_t bytes)
{
    const size_t q = bytes >= ((size_t)1 << 24) ? ((size_t)1 << 21) : 256;  // 2 MiB steps for big blocks
    return (bytes + q - 1) / q * q;
}

// Caller holds c.mu.  Drops one block's reference to its free event.
void drop_event(DeviceCache& c, FreeEvent* f)
{
    if (f && --f->refs == 0) {
        c.events.push_back(f->ev);
        delete f;
    }
}

// Caller holds c.mu.  Waits for the idle blocks' frees and returns them.
void release_idle(DeviceCache& c)
{
    for (CachedBlock& b : c.idle) {
        if (b.freed) {
            (void)hipEventSynchronize(b.freed->ev);
            drop_event(c, b.freed);
        }
        (void)hipFree(b.ptr);
    }
    c.idle.clear();
}

hipError_t dev_alloc(void** ptr, size_t bytes, int dev, hipStream_t s)
{
    *ptr = nullptr;
    bytes = round_block(bytes == 0 ? 256 : bytes);
    DeviceCache& c = cache_for(dev);
    std::lock_guard<std::mutex> lk(c.mu);
    int best = -1;
    for (int i = 0; i < (int)c.idle.size(); ++i) {
        const size_t have = c.idle[i].bytes;
        if (have >= bytes && have <= 2 * bytes && (best < 0 || have < c.idle[best].bytes)) best = i;
    }
    if (best >= 0) {
        CachedBlock b = c.idle[best];
        c.idle.erase(c.idle.begin() + best);
        if (b.freed) {
            (void)hipStreamWaitEvent(s, b.freed->ev, 0);
            drop_event(c, b.freed);
        }
        c.live.emplace_back(b.ptr, b.bytes);
        *ptr = b.ptr;
        return hipSuccess;
    }
    hipError_t e = hipMalloc(ptr, bytes);
    if (e == hipErrorOutOfMemory || e == hipErrorMemoryAllocation) {
        (void)hipGetLastError();
        release_idle(c);
        e = hipMalloc(ptr, bytes);
    }
    if (e != hipSuccess) {
        *ptr = nullptr;
        return e;
    }
    c.live.emplace_back(*ptr, bytes);
    return hipSuccess;
}

// Returns blocks to the cache.  Their last uses are ordered on stream s:
// one event recorded there now orders whoever takes any of them next.
// With `idle` the caller has already waited for them (no event).
void dev_free_many(void* const* ptrs, size_t count, int dev, hipStream_t s, bool idle = false)
{
    DeviceCache& c = cache_for(dev);
    std::lock_guard<std::mutex> lk(c.mu);
    FreeEvent* fe = nullptr;
    if (!idle) {
        hipEvent_t ev = nullptr;
        if (!c.events.empty()) {
            ev = c.events.back();
            c.events.pop_back();
        } else if (hipEventCreateWithFlags(&ev, hipEventDisableTiming) != hipSuccess) {
            (void)hipGetLastError();
            ev = nullptr;
        }
        if (ev && hipEventRecord(ev, s) != hipSuccess) {
            (void)hipGetLastError();
            c.events.push_back(ev);
            ev = nullptr;
        }
        if (ev) fe = new FreeEvent{ev, 0};
        else (void)hipStreamSynchronize(s);  // no event: wait here instead
    }
    for (size_t k = 0; k < count; ++k) {
        void* ptr = ptrs[k];
        if (!ptr) continue;
        for (size_t i = 0; i < c.live.size(); ++i) {
            if (c.live[i].first != ptr) continue;
            const size_t bytes = c.live[i].second;
            c.live[i] = c.live.back();
            c.live.pop_back();
            if (fe) ++fe->refs;
            c.idle.push_back(CachedBlock{ptr, bytes, fe});
            break;
        }
    }
    if (fe && fe->refs == 0) {
        c.events.push_back(fe->ev);
        delete fe;
    }
}

void dev_free(void* ptr, int dev, hipStream_t s)
{
    if (ptr) dev_free_many(&ptr, 1, dev, s);
}

// ------------------------------------------------------------- profiling

struct ProfEntry {
    const char* name;
    int64_t launches;
    double total_ms;
};
struct Pending {
    const char* name;
    hipEvent_t a, b;
};
bool g_prof_on = false;
std::string g_prof_only;  // when not empty: the one label bracketed
std::vector<ProfEntry> g_prof;
std::vector<Pending> g_pending;
std::vector<hipEvent_t> g_event_pool;

hipEvent_t take_event()
{
    if (!g_event_pool.empty()) {
        hipEvent_t e = g_event_pool.back();
        g_event_pool.pop_back();
        return e;
    }
    // Timing only: read after the caller has synchronised the device, so the
    // record needs no system-scope fence (a fence per record flushes caches
    // and adds microseconds between short launches).
    hipEvent_t e = nullptr;
    if (hipEventCreateWithFlags(&e, hipEventDisableSystemFence) != hipSuccess) return nullptr;
    return e;
}

}  // namespace

namespace lx {

int prof_begin(const char* name, hipStream_t s)
{
    if (!g_prof_on) return -1;
    if (!g_prof_only.empty() && g_prof_only != name) return -1;
    Pending p{name, take_event(), take_event()};
    if (!p.a || !p.b) return -1;
    (void)hipEventRecord(p.a, s);
    g_pending.push_back(p);
    return (int)g_pending.size() - 1;
}

void prof_end(int token, hipStream_t s)
{
    if (token < 0 || token >= (int)g_pending.size()) return;
    (void)hipEventRecord(g_pending[token].b, s);
}

}  // namespace lx

// ------------------------------------------------------- host-side helpers

// Pinned host words for reading a plan's NaN/Inf flag back: a copy into
// pinned memory is a plain DMA, where pageable memory would be staged.
// One allocation per process, slots handed out under a lock; when all are
// taken, the caller falls back to its own (pageable) word.
struct PinnedFlags {
    std::mutex mu;
    uint32_t* base = nullptr;
    bool tried = false;
    std::vector<int> free;
};
PinnedFlags g_pinned;
constexpr int kPinnedSlots = 256;

uint32_t* take_pinned_flag()
{
    std::lock_guard<std::mutex> lk(g_pinned.mu);
    if (!g_pinned.tried) {
        g_pinned.tried = true;
        void* p = nullptr;
        if (hipHostMalloc(&p, kPinnedSlots * 64, hipHostMallocDefault) == hipSuccess) {
            g_pinned.base = (uint32_t*)p;
            for (int i = kPinnedSlots - 1; i >= 0; --i) g_pinned.free.push_back(i);
        } else {
            (void)hipGetLastError();
        }
    }
    if (g_pinned.free.empty()) return nullptr;
    const int i = g_pinned.free.back();
    g_pinned.free.pop_back();
    return g_pinned.base + (size_t)i * 16;  // one 64-byte line per slot
}

void give_pinned_flag(uint32_t* w)
{
    if (!w) return;
    std::lock_guard<std::mutex> lk(g_pinned.mu);
    g_pinned.free.push_back((int)((w - g_pinned.base) / 16));
}

// LDS bytes a workgroup may use on a device (looked up once per device).
int lds_budget(int dev)
{
    static std::mutex mu;
    static std::vector<int> cached;
    std::lock_guard<std::mutex> lk(mu);
    if ((int)cached.size() <= dev) cached.resize((size_t)dev + 1, 0);
    if (!cached[dev]) {
        int lds = 0;
        if (hipDeviceGetAttribute(&lds, hipDeviceAttributeMaxSharedMemoryPerBlock, dev) != hipSuccess) {
            (void)hipGetLastError();
            lds = 65536;
        }
        if (lds > 160 * 1024) lds = 160 * 1024;
        cached[dev] = lds - 1024;
    }
    return cached[dev];
}

// ----------------------------------------------------------------- plans

struct laplex_plan_s {
    int device = 0;
    int64_t n = 0, k = 0;
    bool sym = true, phased = false;
    int algo = LAPLEX_ALGO_AUTO;
    double temperature = 1.0;
    double inv_t = 1.0;  // 1 / temperature, +inf at temperature 0
    int lds_bytes = 0;
    // sorted sides and the replay records of their sorts
    float* sa = nullptr;
    float* sb = nullptr;  // general only (symmetric: aliases sa)
    lx::SortRecords ra, rb;
    // permutations (rank -> original index), made from the records on demand
    uint32_t* pa = nullptr;
    uint32_t* pb = nullptr;
    // Gram: first sorted-b position of every interval of the sorted a, and
    // the rank of each original index of a, made on the first gram call
    uint32_t* gbound = nullptr;
    uint32_t* grank = nullptr;
    // Gram: b's inputs split by original index into one slice per die
    uint32_t* gslice_off = nullptr;
    uint32_t* gslice_src = nullptr;
    float* gslice_b = nullptr;
    float* gslice_c = nullptr;
    float* gslice_s = nullptr;
    // copies in original order (general only)
    float* a0 = nullptr;
    float* b0 = nullptr;
    float* phi0 = nullptr;
    float* psi0 = nullptr;
    // phase factors by rank: phi by a's order, psi by b's order (a's if symmetric)
    float* cphi = nullptr;
    float* sphi = nullptr;
    float* cpsi = nullptr;
    float* spsi = nullptr;
    // general plans: cos/sin of the phases in original order
    float* cphi0 = nullptr;
    float* sphi0 = nullptr;
    float* cpsi0 = nullptr;
    float* spsi0 = nullptr;
    // plan_create_apply keeps its input x for a later backward: the rows by
    // rank (when they travelled with the sort; stride pad64(n)) or a copy in
    // original order
    float* kept_x = nullptr;
    bool kept_by_rank = false;
    int64_t kept_batch = 0;
    // workspace for apply / gram
    void* ws = nullptr;
    size_t ws_bytes = 0;
    std::vector<void*> owned;
    // the stream the plan's work was ordered on (multi: more than one)
    hipStream_t stream = nullptr;
    bool stream_known = false, multi_stream = false;
};

namespace {

struct DeviceGuard {
    int prev = -1;
    explicit DeviceGuard(int dev)
    {
        if (hipGetDevice(&prev) == hipSuccess && prev != dev) (void)hipSetDevice(dev);
        else prev = -1;
    }
    ~DeviceGuard()
    {
        if (prev >= 0) (void)hipSetDevice(prev);
    }
};

hipError_t plan_alloc(laplex_plan p, void** out, size_t bytes, hipStream_t s)
{
    hipError_t e = dev_alloc(out, bytes, p->device, s);
    if (e == hipSuccess) p->owned.push_back(*out);
    return e;
}

void note_stream(laplex_plan p, hipStream_t s)
{
    if (!p->stream_known) {
        p->stream = s;
        p->stream_known = true;
    } else if (p->stream != s) {
        p->multi_stream = true;
    }
}

void plan_release(laplex_plan p)
{
    if (!p) return;
    std::vector<void*> blocks = p->owned;
    if (p->ws) blocks.push_back(p->ws);
    if (p->stream_known && !p->multi_stream) {
        // all of the plan's work was ordered on one stream: the blocks go
        // back to the cache behind one event on it, nothing waits here
        dev_free_many(blocks.data(), blocks.size(), p->device, p->stream);
    } else {
        // several streams may still use the plan's memory: wait for the
        // device, then the blocks go back to the cache already idle
        (void)hipDeviceSynchronize();
        dev_free_many(blocks.data(), blocks.size(), p->device, nullptr, true);
    }
    delete p;
}

hipError_t ensure_ws(laplex_plan p, size_t bytes, hipStream_t s)
{
    if (p->ws_bytes >= bytes) return hipSuccess;
    if (p->ws) dev_free(p->ws, p->device, s);
    p->ws = nullptr;
    p->ws_bytes = 0;
    const size_t want = align256(bytes + bytes / 8);
    hipError_t e = dev_alloc(&p->ws, want, p->device, s);
    if (e != hipSuccess) {
        (void)hipGetLastError();
        e = dev_alloc(&p->ws, align256(bytes), p->device, s);
        if (e != hipSuccess) return e;
        p->ws_bytes = align256(bytes);
        return hipSuccess;
    }
    p->ws_bytes = want;
    return hipSuccess;
}

bool ranges_overlap(const void* a, size_t na, const void* b, size_t nb)
{
    const char* x = (const char*)a;
    const char* y = (const char*)b;
    return x < y + nb && y < x + na;
}

laplex_status check_device()
{
    int count = 0;
    if (hipGetDeviceCount(&count) != hipSuccess || count <= 0) {
        (void)hipGetLastError();
        return fail(LAPLEX_ERR_NO_DEVICE, "no HIP device visible");
    }
    return LAPLEX_OK;
}



// Bump allocator over the plan workspace.
struct Carve {
    char* base;
    size_t off = 0;
    explicit Carve(void* b) : base((char*)b) {}
    template <class T>
    T* take(size_t count)
    {
        T* p = (T*)(base + off);
        off += align256(count * sizeof(T));
        return p;
    }
};

// Workspace of one scan along a side of length len: `vecs` single-channel
// rows [batch][ld], `chrows` rows per channel [ch][batch][ld], and the tile
// composites and carries.
size_t scan_ws_bytes(int64_t len, int64_t batch, int ch, int vecs, int chrows)
{
    const int64_t ld = pad64(len);
    const int64_t tiles = (len + lx::kScanTile - 1) / lx::kScanTile;
    const int64_t groups = (tiles + lx::kCarryGroup - 1) / lx::kCarryGroup;
    size_t b = 0;
    b += (size_t)vecs * align256((size_t)batch * ld * 4);
    b += (size_t)chrows * align256((size_t)ch * batch * ld * 4);
    b += align256((size_t)ch * batch * tiles * 4 * 8);
    b += align256((size_t)ch * batch * groups * 4 * 8);
    b += align256((size_t)ch * batch * tiles * 2 * 8);
    return b;
}

void scan_common(lx::ScanArgs& A, Carve& cv, int64_t len, int64_t batch, int ch)
{
    A.channels = ch;
    A.n = len;
    A.tiles = (len + lx::kScanTile - 1) / lx::kScanTile;
    A.batch = batch;
    A.ld = pad64(len);
    const int64_t groups = (A.tiles + lx::kCarryGroup - 1) / lx::kCarryGroup;
    A.agg = cv.take<double>((size_t)ch * batch * A.tiles * 4);
    A.gagg = cv.take<double>((size_t)ch * batch * groups * 4);
    A.carry = cv.take<double>((size_t)ch * batch * A.tiles * 2);
}

// Sides at least this long move x into sorted order and y back by replaying
// the sort (streaming passes); shorter ones gather/scatter through the
// permutation directly (fewer launches).
int64_t replay_min()
{
    static int64_t v = [] {
        const char* e = getenv("LAPLEX_REPLAY_MIN");
        return e ? atoll(e) : (int64_t)1 << 20;
    }();
    return v;
}

// Make the permutation of side 0 (a) or 1 (b) from the sort records.
hipError_t ensure_perm(laplex_plan p, int side, hipStream_t s)
{
    uint32_t** dst = side == 0 ? &p->pa : &p->pb;
    if (*dst) return hipSuccess;
    if (side == 1 && p->sym) {
        hipError_t e = ensure_perm(p, 0, s);
        p->pb = p->pa;
        return e;
    }
    const lx::SortRecords& R = side == 0 ? p->ra : p->rb;
    void* perm = nullptr;
    void* tmp = nullptr;
    hipError_t e = plan_alloc(p, &perm, (size_t)R.n * 4, s);
    if (e != hipSuccess) return e;
    e = dev_alloc(&tmp, (size_t)R.n * 4, p->device, s);
    if (e != hipSuccess) return e;
    e = lx::perm_from_records(R, (uint32_t*)perm, (uint32_t*)tmp, s);
    dev_free(tmp, p->device, s);
    if (e == hipSuccess) *dst = (uint32_t*)perm;
    return e;
}

}  // namespace

extern "C" {

const char* laplex_status_str(laplex_status s)
{
    switch (s) {
        case LAPLEX_OK: return "ok";
        case LAPLEX_ERR_INVALID_ARGUMENT: return "invalid argument";
        case LAPLEX_ERR_NONFINITE_ANCHOR: return "non-finite anchor or phase";
        case LAPLEX_ERR_OUT_OF_MEMORY: return "out of device memory";
        case LAPLEX_ERR_UNSUPPORTED: return "unsupported";
        case LAPLEX_ERR_DEVICE: return "device error";
        case LAPLEX_ERR_NO_DEVICE: return "no device";
    }
    return "unknown status";
}

const char* laplex_last_error(void) { return g_last_error.c_str(); }

namespace {

// Plan creation; with x != NULL (symmetric plans only) also y = K x, sorting
// the rows of x along with the anchors when the plan replays its sort.
laplex_status plan_create_impl(laplex_plan* out, const float* a, int64_t n, const float* b, int64_t k,
                               const float* phi, const float* psi, const float* x, float* y, int64_t batch,
                               void* stream)
{
    if (out) *out = nullptr;
    if (!out) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "out is NULL");
    if (!a) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "a is NULL");
    if (n < 1 || n > kMaxLen) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "n must be in [1, 2^30]");
    const bool sym = b == nullptr;
    if (sym && k != 0 && k != n) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "symmetric plan: k must be 0 or n");
    if (!sym && (k < 1 || k > kMaxLen)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "k must be in [1, 2^30]");
    if ((phi == nullptr) != (psi == nullptr))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "phi and psi: give both or neither");
    if (sym) k = n;
    laplex_status st = check_device();
    if (st != LAPLEX_OK) return st;

    hipStream_t s = (hipStream_t)stream;
    laplex_plan p = new laplex_plan_s();
    note_stream(p, s);
    p->n = n;
    p->k = k;
    p->sym = sym;
    p->phased = phi != nullptr;
    void* scratch = nullptr;
    uint32_t* flag = nullptr;
    uint32_t own_flag = 0;
    uint32_t* pinned = take_pinned_flag();
    uint32_t* host_flag = pinned ? pinned : &own_flag;
    struct PinnedRelease {
        uint32_t* w;
        ~PinnedRelease() { give_pinned_flag(w); }
    } pinned_release{pinned};
    auto bail = [&](laplex_status code) {
        if (scratch) dev_free(scratch, p->device, s);
        plan_release(p);
        return code;
    };
#define LX_PLAN_TRY(call, where)                                  \
    do {                                                         \
        const laplex_status lx_s2_ = from_hip((call), (where));  \
        if (lx_s2_ != LAPLEX_OK) return bail(lx_s2_);            \
    } while (0)

    LX_PLAN_TRY(hipGetDevice(&p->device), "hipGetDevice");
    p->lds_bytes = lds_budget(p->device);
    LX_PLAN_TRY(plan_alloc(p, (void**)&flag, 256, s), "alloc flag");
    LX_PLAN_TRY(plan_alloc(p, (void**)&p->sa, (size_t)n * 4, s), "alloc sorted a");
    const bool small_plan = sym && n <= lx::kSmallMax && n < replay_min();
    // the small plan kernel writes the flag whole; the others OR into it
    if (!small_plan) LX_PLAN_TRY(lx::fill_u32(flag, 0u, 1, s), "clear flag");
    if (small_plan) {
        // A small symmetric plan in one workgroup: the sorted anchors, the
        // permutation (the sort records are never needed below the replay
        // size) and the phase factors by rank; y = K x too for a few vectors.
        LX_PLAN_TRY(plan_alloc(p, (void**)&p->pa, (size_t)n * 4, s), "alloc permutation");
        p->sb = p->sa;
        p->pb = p->pa;
        if (p->phased) {
            LX_PLAN_TRY(plan_alloc(p, (void**)&p->cphi, (size_t)n * 4, s), "alloc phases");
            LX_PLAN_TRY(plan_alloc(p, (void**)&p->sphi, (size_t)n * 4, s), "alloc phases");
            LX_PLAN_TRY(plan_alloc(p, (void**)&p->cpsi, (size_t)n * 4, s), "alloc phases");
            LX_PLAN_TRY(plan_alloc(p, (void**)&p->spsi, (size_t)n * 4, s), "alloc phases");
        }
        const bool with_y = x != nullptr && batch <= 8;
        // the kernel that computes y also copies x for a later backward
        float* keep = nullptr;
        if (with_y) LX_PLAN_TRY(plan_alloc(p, (void**)&keep, (size_t)(batch * n) * 4, s), "alloc kept x");
        lx::SmallSymArgs S;
        S.n = n;
        S.batch = with_y ? (int)batch : 0;
        S.inv_t = p->inv_t;
        S.a = a;
        S.phi = phi;
        S.psi = psi;
        S.x = with_y ? x : nullptr;
        S.x_keep = keep;
        S.y = with_y ? y : nullptr;
        S.sa = p->sa;
        S.perm = p->pa;
        S.cphi = p->cphi;
        S.sphi = p->sphi;
        S.cpsi = p->cpsi;
        S.spsi = p->spsi;
        S.flag = flag;
        LX_PLAN_TRY(lx::small_sym_launch(S, s), "small plan");
        LX_PLAN_TRY(hipMemcpyAsync(host_flag, flag, 4, hipMemcpyDeviceToHost, s), "read flag");
        LX_PLAN_TRY(hipStreamSynchronize(s), "synchronize");
        if (*host_flag & 1u) return bail(fail(LAPLEX_ERR_NONFINITE_ANCHOR, "NaN or Inf among anchors or phases"));
        if (x) {
            // x in its original order is kept for a later backward (copied
            // by the plan kernel when it computed y)
            laplex_status st2 = with_y ? LAPLEX_OK : laplex_apply(p, x, y, batch, 0, stream);
            if (!with_y && st2 == LAPLEX_OK)
                st2 = from_hip(plan_alloc(p, (void**)&keep, (size_t)(batch * n) * 4, s), "alloc kept x");
            if (!with_y && st2 == LAPLEX_OK)
                st2 = from_hip(hipMemcpyAsync(keep, x, (size_t)(batch * n) * 4, hipMemcpyDeviceToDevice, s), "copy x");
            p->kept_x = keep;
            p->kept_by_rank = false;
            p->kept_batch = batch;
            if (st2 != LAPLEX_OK) {
                plan_release(p);
                return st2;
            }
        }
        *out = p;
        return LAPLEX_OK;
    }
    {
        void* rec = nullptr;
        LX_PLAN_TRY(plan_alloc(p, &rec, lx::sort_record_bytes(n), s), "alloc sort records");
        p->ra = lx::sort_records_at(rec, n);
    }
    const int64_t big = sym ? n : (n > k ? n : k);
    // Symmetric plans on the replay path sort value rows with the anchors:
    // the rows of x (when applying at once) and the phases.
    const bool replay = sym && n >= replay_min();
    const int ph_rows = p->phased ? 2 : 0;
    const bool fuse = x != nullptr && replay && batch + ph_rows <= lx::kMaxSortVals;
    lx::SortVals V;
    if (replay) {
        if (fuse)
            for (int64_t v = 0; v < batch; ++v) V.in[V.rows++] = x + v * n;
        if (p->phased) {
            V.in[V.rows++] = phi;
            V.in[V.rows++] = psi;
        }
        V.ld = pad64(n);
    }
    const size_t vbytes = align256((size_t)V.rows * V.ld * 4);
    // value buffers: va and vb for the sort; when applying at once the sorted
    // rows (vb) stay with the plan for a later backward, and a third buffer
    // joins the ping-pong of the replay back into y
    LX_PLAN_TRY(dev_alloc(&scratch, lx::sort_scratch_bytes(big, V.rows > 0) + 2 * vbytes, p->device, s),
                "alloc sort scratch");
    float* vt = nullptr;
    if (V.rows) {
        V.va = (float*)((char*)scratch + lx::sort_scratch_bytes(big, V.rows > 0));
        if (fuse) {
            LX_PLAN_TRY(plan_alloc(p, (void**)&V.vb, vbytes, s), "alloc kept x");
            vt = (float*)((char*)V.va + vbytes);
            p->kept_x = V.vb;
            p->kept_by_rank = true;
            p->kept_batch = batch;
        } else {
            V.vb = (float*)((char*)V.va + vbytes);
        }
    }
    LX_PLAN_TRY(lx::sort_launch(a, n, p->sa, p->ra, scratch, flag, s, V.rows ? &V : nullptr), "sort a");
    if (sym) {
        p->sb = p->sa;
        p->rb = p->ra;
        // short sides gather through the permutation
        if (!replay) LX_PLAN_TRY(ensure_perm(p, 0, s), "permutation");
        if (p->phased) {
            LX_PLAN_TRY(plan_alloc(p, (void**)&p->cphi, (size_t)n * 4, s), "alloc phases");
            LX_PLAN_TRY(plan_alloc(p, (void**)&p->sphi, (size_t)n * 4, s), "alloc phases");
            LX_PLAN_TRY(plan_alloc(p, (void**)&p->cpsi, (size_t)n * 4, s), "alloc phases");
            LX_PLAN_TRY(plan_alloc(p, (void**)&p->spsi, (size_t)n * 4, s), "alloc phases");
            if (replay) {
                // the phases came out of the sort in rank order: the last two rows
                const float* sphi_rank = V.vb + (V.rows - 2) * V.ld;
                const float* spsi_rank = V.vb + (V.rows - 1) * V.ld;
                LX_PLAN_TRY(lx::phase_factors_launch(sphi_rank, nullptr, n, p->cphi, p->sphi, flag, s), "phi factors");
                LX_PLAN_TRY(lx::phase_factors_launch(spsi_rank, nullptr, n, p->cpsi, p->spsi, flag, s), "psi factors");
            } else {
                LX_PLAN_TRY(lx::phase_factors_launch(phi, p->pa, n, p->cphi, p->sphi, flag, s), "phi factors");
                LX_PLAN_TRY(lx::phase_factors_launch(psi, p->pa, n, p->cpsi, p->spsi, flag, s), "psi factors");
            }
        }
        if (fuse) {
            // y = K x from the sorted rows of x: scan in place, replay back into y
            const int ch = p->phased ? 2 : 1;
            LX_PLAN_TRY(ensure_ws(p, scan_ws_bytes(n, batch, ch, 0, 0), s), "workspace");
            Carve cv(p->ws);
            lx::ScanArgs A;
            A.mode = lx::kScanSym;
            scan_common(A, cv, n, batch, ch);
            A.inv_t = p->inv_t;
            A.s = p->sa;
            A.random = false;
            A.xs = V.vb;  // kept: y by rank goes to va
            A.ys = V.va;
            if (p->phased) {
                A.in_c = p->cpsi;
                A.in_s = p->spsi;
                A.out_c = p->cphi;
                A.out_s = p->sphi;
            }
            LX_PLAN_TRY(lx::scan_launch(A, s), "symmetric apply");
            const lx::SortRecords& R = p->ra;
            LX_PLAN_TRY(lx::replay_launch(R, 3, false, V.va, V.ld, vt, V.ld, batch, s), "replay");
            LX_PLAN_TRY(lx::replay_launch(R, 2, false, vt, V.ld, V.va, V.ld, batch, s), "replay");
            LX_PLAN_TRY(lx::replay_launch(R, 1, false, V.va, V.ld, vt, V.ld, batch, s), "replay");
            LX_PLAN_TRY(lx::replay_launch(R, 0, false, vt, V.ld, y, n, batch, s), "replay");
        }
    } else {
        LX_PLAN_TRY(plan_alloc(p, (void**)&p->sb, (size_t)k * 4, s), "alloc sorted b");
        {
            void* rec = nullptr;
            LX_PLAN_TRY(plan_alloc(p, &rec, lx::sort_record_bytes(k), s), "alloc sort records");
            p->rb = lx::sort_records_at(rec, k);
        }
        LX_PLAN_TRY(lx::sort_launch(b, k, p->sb, p->rb, scratch, flag, s), "sort b");
        LX_PLAN_TRY(ensure_perm(p, 0, s), "permutation of a");
        LX_PLAN_TRY(ensure_perm(p, 1, s), "permutation of b");
        LX_PLAN_TRY(plan_alloc(p, (void**)&p->a0, (size_t)n * 4, s), "alloc a copy");
        LX_PLAN_TRY(plan_alloc(p, (void**)&p->b0, (size_t)k * 4, s), "alloc b copy");
        LX_PLAN_TRY(hipMemcpyAsync(p->a0, a, (size_t)n * 4, hipMemcpyDeviceToDevice, s), "copy a");
        LX_PLAN_TRY(hipMemcpyAsync(p->b0, b, (size_t)k * 4, hipMemcpyDeviceToDevice, s), "copy b");
        if (p->phased) {
            LX_PLAN_TRY(plan_alloc(p, (void**)&p->phi0, (size_t)n * 4, s), "alloc phases");
            LX_PLAN_TRY(plan_alloc(p, (void**)&p->psi0, (size_t)k * 4, s), "alloc phases");
            LX_PLAN_TRY(plan_alloc(p, (void**)&p->cphi, (size_t)n * 4, s), "alloc phases");
            LX_PLAN_TRY(plan_alloc(p, (void**)&p->sphi, (size_t)n * 4, s), "alloc phases");
            LX_PLAN_TRY(plan_alloc(p, (void**)&p->cpsi, (size_t)k * 4, s), "alloc phases");
            LX_PLAN_TRY(plan_alloc(p, (void**)&p->spsi, (size_t)k * 4, s), "alloc phases");
            LX_PLAN_TRY(hipMemcpyAsync(p->phi0, phi, (size_t)n * 4, hipMemcpyDeviceToDevice, s), "copy phi");
            LX_PLAN_TRY(hipMemcpyAsync(p->psi0, psi, (size_t)k * 4, hipMemcpyDeviceToDevice, s), "copy psi");
            LX_PLAN_TRY(lx::phase_factors_launch(phi, p->pa, n, p->cphi, p->sphi, flag, s), "phi factors");
            LX_PLAN_TRY(lx::phase_factors_launch(psi, p->pb, k, p->cpsi, p->spsi, flag, s), "psi factors");
            LX_PLAN_TRY(plan_alloc(p, (void**)&p->cphi0, (size_t)n * 4, s), "alloc phases");
            LX_PLAN_TRY(plan_alloc(p, (void**)&p->sphi0, (size_t)n * 4, s), "alloc phases");
            LX_PLAN_TRY(plan_alloc(p, (void**)&p->cpsi0, (size_t)k * 4, s), "alloc phases");
            LX_PLAN_TRY(plan_alloc(p, (void**)&p->spsi0, (size_t)k * 4, s), "alloc phases");
            LX_PLAN_TRY(lx::phase_factors_launch(phi, nullptr, n, p->cphi0, p->sphi0, flag, s), "phi factors");
            LX_PLAN_TRY(lx::phase_factors_launch(psi, nullptr, k, p->cpsi0, p->spsi0, flag, s), "psi factors");
        }
    }
    dev_free(scratch, p->device, s);
    scratch = nullptr;
    LX_PLAN_TRY(hipMemcpyAsync(host_flag, flag, 4, hipMemcpyDeviceToHost, s), "read flag");
    LX_PLAN_TRY(hipStreamSynchronize(s), "synchronize");
    if (*host_flag & 1u) return bail(fail(LAPLEX_ERR_NONFINITE_ANCHOR, "NaN or Inf among anchors or phases"));
#undef LX_PLAN_TRY
    if (x && !fuse) {
        // not fused (short side or too many rows): the plain apply, and a copy
        // of x kept for a later backward
        laplex_status st2 = laplex_apply(p, x, y, batch, 0, stream);
        if (st2 == LAPLEX_OK) {
            float* keep = nullptr;
            st2 = from_hip(plan_alloc(p, (void**)&keep, (size_t)(batch * n) * 4, s), "alloc kept x");
            if (st2 == LAPLEX_OK)
                st2 = from_hip(hipMemcpyAsync(keep, x, (size_t)(batch * n) * 4, hipMemcpyDeviceToDevice, s), "copy x");
            p->kept_x = keep;
            p->kept_by_rank = false;
            p->kept_batch = batch;
        }
        if (st2 != LAPLEX_OK) {
            plan_release(p);
            return st2;
        }
    }
    *out = p;
    return LAPLEX_OK;
}

}  // namespace

laplex_status laplex_plan_create(laplex_plan* out, const float* a, int64_t n, const float* b, int64_t k,
                                 const float* phi, const float* psi, void* stream)
{
    return plan_create_impl(out, a, n, b, k, phi, psi, nullptr, nullptr, 0, stream);
}

laplex_status laplex_plan_create_apply(laplex_plan* out, const float* a, int64_t n, const float* phi,
                                       const float* psi, const float* x, float* y, int64_t batch, void* stream)
{
    if (out) *out = nullptr;
    if (!out) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "out is NULL");
    if (!x || !y) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "x or y is NULL");
    if (batch < 1) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "batch must be >= 1");
    if (n >= 1 && (batch > (int64_t)1 << 40 || (double)batch * (double)n > 4.0e18 / 4))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "batch too large");
    if (n >= 1 && ranges_overlap(x, (size_t)(batch * n) * 4, y, (size_t)(batch * n) * 4))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "x and y overlap");
    return plan_create_impl(out, a, n, nullptr, 0, phi, psi, x, y, batch, stream);
}

laplex_status laplex_plan_destroy(laplex_plan p)
{
    if (!p) return LAPLEX_OK;
    DeviceGuard g(p->device);
    plan_release(p);
    return LAPLEX_OK;
}

laplex_status laplex_plan_perm(laplex_plan p, int side, const uint32_t** perm_dev)
{
    if (!p || !perm_dev || (side != 0 && side != 1)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "bad plan_perm arguments");
    DeviceGuard g(p->device);
    note_stream(p, nullptr);
    LX_TRY(ensure_perm(p, side, nullptr), "permutation");
    LX_TRY(hipStreamSynchronize(nullptr), "synchronize");
    *perm_dev = side == 0 ? p->pa : p->pb;
    return LAPLEX_OK;
}

laplex_status laplex_plan_sorted(laplex_plan p, int side, const float** sorted_dev)
{
    if (!p || !sorted_dev || (side != 0 && side != 1))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "bad plan_sorted arguments");
    *sorted_dev = side == 0 ? p->sa : p->sb;
    return LAPLEX_OK;
}

laplex_status laplex_plan_info(laplex_plan p, int64_t* n, int64_t* k, int* flags)
{
    if (!p) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "plan is NULL");
    if (n) *n = p->n;
    if (k) *k = p->k;
    if (flags) *flags = (p->sym ? LAPLEX_PLAN_SYMMETRIC : 0) | (p->phased ? LAPLEX_PLAN_PHASED : 0);
    return LAPLEX_OK;
}

laplex_status laplex_plan_set_option(laplex_plan p, int option, int64_t value)
{
    if (!p) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "plan is NULL");
    if (option != LAPLEX_OPT_GENERAL_ALGO) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "unknown option");
    if (value != LAPLEX_ALGO_AUTO && value != LAPLEX_ALGO_BUCKET && value != LAPLEX_ALGO_EVALUATE)
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "unknown algorithm");
    p->algo = (int)value;
    return LAPLEX_OK;
}

laplex_status laplex_plan_set_temperature(laplex_plan p, double t)
{
    if (!p) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "plan is NULL");
    if (!(t == 0.0 || (t >= (double)FLT_MIN && t <= (double)FLT_MAX)))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "temperature must be 0 or in [FLT_MIN, FLT_MAX]");
    p->temperature = t;
    p->inv_t = t > 0.0 ? 1.0 / t : HUGE_VAL;
    return LAPLEX_OK;
}

}  // extern "C"

namespace {

// Where an apply takes its workspace: the plan's own (grown on demand), or
// a fixed region that must already be large enough (no allocation).
struct WsSource {
    void* fixed = nullptr;
    size_t fixed_bytes = 0;
};

laplex_status take_ws(laplex_plan p, size_t need, hipStream_t s, const WsSource& src, void** base)
{
    if (src.fixed) {
        if (need > src.fixed_bytes)
            return fail(LAPLEX_ERR_INVALID_ARGUMENT, "this apply needs " + std::to_string(need) +
                                                         " bytes of scratch; the fixed scratch holds " +
                                                         std::to_string(src.fixed_bytes));
        *base = src.fixed;
        return LAPLEX_OK;
    }
    LX_TRY(ensure_ws(p, need, s), "workspace");
    *base = p->ws;
    return LAPLEX_OK;
}

#define LX_WS(need, base)                                           \
    do {                                                            \
        const laplex_status lx_w_ = take_ws(p, (need), s, src, &(base)); \
        if (lx_w_ != LAPLEX_OK) return lx_w_;                       \
    } while (0)

laplex_status apply_impl(laplex_plan p, const float* x, float* y, int64_t batch, int transpose, void* stream,
                         const WsSource& src)
{
    if (!p) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "plan is NULL");
    if (!x || !y) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "x or y is NULL");
    if (batch < 1) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "batch must be >= 1");
    if (transpose != 0 && transpose != 1) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "transpose must be 0 or 1");
    const int64_t len_in = transpose ? p->n : p->k;
    const int64_t len_out = transpose ? p->k : p->n;
    if (batch > (int64_t)1 << 40 || (double)batch * (double)(len_in > len_out ? len_in : len_out) > 4.0e18 / 4)
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "batch too large");
    if (ranges_overlap(x, (size_t)(batch * len_in) * 4, y, (size_t)(batch * len_out) * 4))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "x and y overlap");
    DeviceGuard g(p->device);
    hipStream_t s = (hipStream_t)stream;
    note_stream(p, s);
    const int ch = p->phased ? 2 : 1;

    if (p->sym) {
        const int64_t n = p->n;
        const bool replay = n >= replay_min();
        if (!replay && !p->pa) {
            if (src.fixed) return fail(LAPLEX_ERR_UNSUPPORTED, "the plan has no permutation yet");
            LX_TRY(ensure_perm(p, 0, s), "permutation");
        }
        void* wsb = nullptr;
        LX_WS(scan_ws_bytes(n, batch, ch, replay ? 2 : 1, 0), wsb);
        Carve cv(wsb);
        lx::ScanArgs A;
        A.mode = lx::kScanSym;
        scan_common(A, cv, n, batch, ch);
        A.inv_t = p->inv_t;
        A.s = p->sa;
        A.perm = p->pa;
        if (p->phased) {
            // K = LAPLEX(a, phi; a, psi): inputs carry psi, outputs phi; K^T swaps them
            A.in_c = transpose ? p->cphi : p->cpsi;
            A.in_s = transpose ? p->sphi : p->spsi;
            A.out_c = transpose ? p->cpsi : p->cphi;
            A.out_s = transpose ? p->spsi : p->sphi;
        }
        if (!replay) {
            A.random = true;
            A.x = x;
            A.y = y;
            A.xs = cv.take<float>((size_t)batch * A.ld);
            LX_TRY(lx::scan_launch(A, s), "symmetric apply");
            return LAPLEX_OK;
        }
        // x -> sorted order by replaying the four radix passes, scan in place,
        // then replay them backwards into y.
        float* t1 = cv.take<float>((size_t)batch * A.ld);
        float* t2 = cv.take<float>((size_t)batch * A.ld);
        const lx::SortRecords& R = p->ra;
        LX_TRY(lx::replay_launch(R, 0, true, x, n, t1, A.ld, batch, s), "replay");
        LX_TRY(lx::replay_launch(R, 1, true, t1, A.ld, t2, A.ld, batch, s), "replay");
        LX_TRY(lx::replay_launch(R, 2, true, t2, A.ld, t1, A.ld, batch, s), "replay");
        LX_TRY(lx::replay_launch(R, 3, true, t1, A.ld, t2, A.ld, batch, s), "replay");
        A.random = false;
        A.xs = t2;
        A.ys = t2;
        LX_TRY(lx::scan_launch(A, s), "symmetric apply");
        LX_TRY(lx::replay_launch(R, 3, false, t2, A.ld, t1, A.ld, batch, s), "replay");
        LX_TRY(lx::replay_launch(R, 2, false, t1, A.ld, t2, A.ld, batch, s), "replay");
        LX_TRY(lx::replay_launch(R, 1, false, t2, A.ld, t1, A.ld, batch, s), "replay");
        LX_TRY(lx::replay_launch(R, 0, false, t1, A.ld, y, n, batch, s), "replay");
        return LAPLEX_OK;
    }

    // General case: side "o" receives the outputs, side "i" holds the inputs.
    const bool out_is_a = transpose == 0;
    const int64_t no = out_is_a ? p->n : p->k;
    const int64_t ni = out_is_a ? p->k : p->n;
    const float* s_o = out_is_a ? p->sa : p->sb;
    const uint32_t* p_o = out_is_a ? p->pa : p->pb;
    const float* s_i = out_is_a ? p->sb : p->sa;
    const uint32_t* p_i = out_is_a ? p->pb : p->pa;
    const float* anchor_o = out_is_a ? p->a0 : p->b0;
    const float* anchor_i = out_is_a ? p->b0 : p->a0;
    const float* co0 = out_is_a ? p->cphi0 : p->cpsi0;  // cos/sin of phases, original order
    const float* so0 = out_is_a ? p->sphi0 : p->spsi0;
    const float* ci0 = out_is_a ? p->cpsi0 : p->cphi0;
    const float* si0 = out_is_a ? p->spsi0 : p->sphi0;
    const float* c_o = out_is_a ? p->cphi : p->cpsi;
    const float* sn_o = out_is_a ? p->sphi : p->spsi;
    const float* c_i = out_is_a ? p->cpsi : p->cphi;
    const float* sn_i = out_is_a ? p->spsi : p->sphi;
    int algo = p->algo;
    if (algo == LAPLEX_ALGO_AUTO) algo = ni <= no ? LAPLEX_ALGO_EVALUATE : LAPLEX_ALGO_BUCKET;

    if (algo == LAPLEX_ALGO_EVALUATE) {
        void* wsb = nullptr;
        LX_WS(scan_ws_bytes(ni, batch, ch, 1, 2), wsb);
        Carve cv(wsb);
        lx::ScanArgs A;
        A.mode = lx::kScanPLPR;
        A.random = true;
        scan_common(A, cv, ni, batch, ch);
        A.inv_t = p->inv_t;
        A.s = s_i;
        A.perm = p_i;
        A.x = x;
        A.xs = cv.take<float>((size_t)batch * A.ld);
        A.pl = cv.take<float>((size_t)ch * batch * A.ld);
        A.pr = cv.take<float>((size_t)ch * batch * A.ld);
        if (p->phased) {
            A.in_c = c_i;
            A.in_s = sn_i;
        }
        LX_TRY(lx::scan_launch(A, s), "scan over the input side");
        lx::EvalArgs E;
        E.channels = ch;
        E.n_out = no;
        E.n_in = ni;
        E.batch = batch;
        E.inv_t = (float)p->inv_t;
        E.out_anchor = anchor_o;
        if (p->phased) {
            E.out_cos = co0;
            E.out_sin = so0;
        }
        E.s_in = s_i;
        E.ld = A.ld;
        E.pl = A.pl;
        E.pr = A.pr;
        E.y = y;
        E.lds_bytes = p->lds_bytes;
        LX_TRY(lx::eval_launch(E, s), "evaluate outputs");
        return LAPLEX_OK;
    }

    // BUCKET: inputs into the intervals of the sorted output side, then scan it.
    lx::BucketArgs Bk;
    Bk.channels = ch;
    Bk.n_out = no;
    Bk.n_in = ni;
    Bk.batch = batch;
    Bk.inv_t = (float)p->inv_t;
    Bk.s_out = s_o;
    Bk.in_anchor = anchor_i;
    if (p->phased) {
        Bk.in_cos = ci0;
        Bk.in_sin = si0;
    }
    Bk.x = x;
    Bk.ld = pad64(no);
    Bk.lds_bytes = p->lds_bytes;
    Bk.partial_floats = lx::bucket_partial_floats(Bk, nullptr, nullptr);
    // a short output side bins in LDS; a long one merges the sorted sides
    const bool merge = Bk.partial_floats == 0;
    const size_t layout_bytes = merge ? 0 : (size_t)lx::bucket_layout_bytes(Bk);
    const size_t need = scan_ws_bytes(no, batch, ch, 0, 2) +
                        (merge ? lx::merge_ws_bytes(ni, no, batch, ch)
                               : align256((size_t)Bk.partial_floats * 4) + align256(layout_bytes));
    void* wsb = nullptr;
    LX_WS(need, wsb);
    Carve cv(wsb);
    lx::ScanArgs A;
    A.mode = lx::kScanUV;
    A.random = true;
    scan_common(A, cv, no, batch, ch);
    A.inv_t = p->inv_t;
    A.s = s_o;
    A.perm = p_o;
    float* u = cv.take<float>((size_t)ch * batch * A.ld);
    float* v = cv.take<float>((size_t)ch * batch * A.ld);
    A.u = u;
    A.v = v;
    A.y = y;
    if (p->phased) {
        A.out_c = c_o;
        A.out_s = sn_o;
    }
    if (merge) {
        lx::MergeArgs M;
        M.channels = ch;
        M.n_out = no;
        M.n_in = ni;
        M.batch = batch;
        M.inv_t = p->inv_t;
        M.s_out = s_o;
        M.s_in = s_i;
        M.perm_in = p_i;
        if (p->phased) {
            M.in_c = c_i;
            M.in_s = sn_i;
        }
        M.x = x;
        M.ld = A.ld;
        M.u = u;
        M.v = v;
        const int64_t tiles = lx::merge_tiles(ni, no);
        M.split = cv.take<uint2>((size_t)tiles + 1);
        M.head = cv.take<double>((size_t)ch * batch * tiles * 2);
        M.tail = cv.take<double>((size_t)ch * batch * tiles * 2);
        LX_TRY(lx::merge_launch(M, s), "merge inputs");
    } else {
        Bk.u = u;
        Bk.v = v;
        Bk.partial = cv.take<float>((size_t)Bk.partial_floats);
        Bk.layout = (void*)cv.take<char>(layout_bytes);
        LX_TRY(lx::bucket_launch(Bk, s), "bucket inputs");
    }
    LX_TRY(lx::scan_launch(A, s), "scan over the output side");
    return LAPLEX_OK;
}

#undef LX_WS

// ------------------------------------------------------ allocation-free apply
//
// laplex_apply_noalloc takes its workspace from this file-scope array, one
// copy per device, kept until the process ends.  Host code reaches it only
// through the device address hipGetSymbolAddress returns (looked up once per
// device, with that device current); the array's own name is a host-side
// stand-in.  Kernels never need it cleared: every word a kernel reads was
// written earlier in the same call.
constexpr size_t kNoAllocBytes = LAPLEX_NOALLOC_SCRATCH_BYTES;
__device__ __align__(256) unsigned char scratch[kNoAllocBytes];

std::mutex g_scratch_mu;
std::vector<void*> g_scratch_ptr;  // per device; null until looked up

hipError_t noalloc_scratch(int dev, void** out)
{
    std::lock_guard<std::mutex> lk(g_scratch_mu);
    if ((int)g_scratch_ptr.size() <= dev) g_scratch_ptr.resize((size_t)dev + 1, nullptr);
    if (!g_scratch_ptr[dev]) {
        void* ptr = nullptr;
        const hipError_t e = hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch));
        if (e != hipSuccess) return e;
        g_scratch_ptr[dev] = ptr;
    }
    *out = g_scratch_ptr[dev];
    return hipSuccess;
}

}  // namespace

extern "C" {

laplex_status laplex_apply(laplex_plan p, const float* x, float* y, int64_t batch, int transpose, void* stream)
{
    return apply_impl(p, x, y, batch, transpose, stream, WsSource{});
}

laplex_status laplex_apply_noalloc(laplex_plan p, const float* x, float* y, int64_t batch, int transpose,
                                   void* stream)
{
    if (!p) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "plan is NULL");
    DeviceGuard g(p->device);
    WsSource src;
    LX_TRY(noalloc_scratch(p->device, &src.fixed), "scratch address");
    src.fixed_bytes = kNoAllocBytes;
    return apply_impl(p, x, y, batch, transpose, stream, src);
}

}  // extern "C"

namespace {

// One side of a general plan's gradient: outputs on side "o" (original
// order) from the prefix/suffix tables of the sorted side "i" of input V.
struct GradSide {
    int64_t no, ni;
    const float* s_i;
    const uint32_t* p_i;
    const float* c_i;   // cos/sin of side i's phases by rank (phased)
    const float* sn_i;
    const float* anchor_o;
    const float* c_o0;  // cos/sin of side o's phases, original order (phased)
    const float* s_o0;
    const float* s_o;       // side o sorted, and its permutation (rank -> original index)
    const uint32_t* p_o;
    const float* anchor_i0; // side i's anchors and phase factors, original order
    const float* c_i0;
    const float* s_i0;
};

// Outputs on a small side (at most 1024 anchors) from a large input side:
// the inputs are bucketed into the intervals of the sorted outputs, in
// their original order (no gather, no tables over the large side).
laplex_status grad_small_side(laplex_plan p, const GradSide& G, const float* V, const float* W, int64_t batch,
                              float* y, float* d_anchor, float* d_phase, hipStream_t s, bool* done)
{
    *done = false;
    const int ch = p->phased ? 2 : 1;
    lx::BucketArgs Bk;
    Bk.channels = ch;
    Bk.n_out = G.no;
    Bk.n_in = G.ni;
    Bk.batch = batch;
    Bk.inv_t = (float)p->inv_t;
    Bk.s_out = G.s_o;
    Bk.in_anchor = G.anchor_i0;
    if (p->phased) {
        Bk.in_cos = G.c_i0;
        Bk.in_sin = G.s_i0;
    }
    Bk.x = V;
    Bk.ld = pad64(G.no);
    Bk.lds_bytes = p->lds_bytes;
    Bk.ties = true;
    Bk.partial_floats = lx::bucket_partial_floats(Bk, nullptr, nullptr);
    if (Bk.partial_floats == 0) return LAPLEX_OK;  // not the LDS-binned shape: the table path instead
    const size_t rows = (size_t)ch * batch * Bk.ld;
    const size_t layout_bytes = (size_t)lx::bucket_layout_bytes(Bk);
    const size_t need = scan_ws_bytes(G.no, batch, ch, 0, 2) + 3 * align256(rows * 4) +
                        align256((size_t)Bk.partial_floats * 4) + align256(layout_bytes);
    LX_TRY(ensure_ws(p, need, s), "workspace");
    Carve cv(p->ws);
    lx::ScanArgs A;
    A.mode = lx::kScanUVLR;
    A.random = false;
    scan_common(A, cv, G.no, batch, ch);
    A.inv_t = p->inv_t;
    A.s = G.s_o;
    float* u = cv.take<float>(rows);
    float* v = cv.take<float>(rows);
    float* tie = cv.take<float>(rows);
    A.u = u;
    A.v = v;
    A.pl = cv.take<float>((size_t)ch * batch * A.ld);
    A.pr = cv.take<float>((size_t)ch * batch * A.ld);
    Bk.u = u;
    Bk.v = v;
    Bk.tie = tie;
    Bk.partial = cv.take<float>((size_t)Bk.partial_floats);
    Bk.layout = cv.take<char>(layout_bytes);
    LX_TRY(lx::bucket_launch(Bk, s), "bucket inputs");
    LX_TRY(lx::scan_launch(A, s), "scan over the output side");
    lx::EvalLRArgs E;
    E.channels = ch;
    E.n_out = G.no;
    E.batch = batch;
    E.ld = A.ld;
    E.anchor_scale = p->temperature > 0.0 ? (float)(-1.0 / p->temperature) : 0.f;
    E.s_out = G.s_o;
    E.perm_out = G.p_o;
    if (p->phased) {
        E.out_cos = G.c_o0;
        E.out_sin = G.s_o0;
    }
    E.L = A.pl;
    E.R = A.pr;
    E.T = tie;
    E.w = W;
    E.y = y;
    E.d_anchor = d_anchor;
    E.d_phase = d_phase;
    LX_TRY(lx::eval_lr_launch(E, s), "evaluate gradients");
    *done = true;
    return LAPLEX_OK;
}

laplex_status grad_general_side(laplex_plan p, const GradSide& G, const float* V, const float* W, int64_t batch,
                                float* y, float* d_anchor, float* d_phase, hipStream_t s)
{
    if (!y && !d_anchor && !d_phase) return LAPLEX_OK;
    if (G.no <= 1024 && G.ni > G.no) {
        bool done = false;
        const laplex_status st = grad_small_side(p, G, V, W, batch, y, d_anchor, d_phase, s, &done);
        if (st != LAPLEX_OK || done) return st;
    }
    const int ch = p->phased ? 2 : 1;
    LX_TRY(ensure_ws(p, scan_ws_bytes(G.ni, batch, ch, 1, 2), s), "workspace");
    Carve cv(p->ws);
    lx::ScanArgs A;
    A.mode = lx::kScanPLPR;
    A.random = true;
    scan_common(A, cv, G.ni, batch, ch);
    A.inv_t = p->inv_t;
    A.s = G.s_i;
    A.perm = G.p_i;
    A.x = V;
    A.xs = cv.take<float>((size_t)batch * A.ld);
    A.pl = cv.take<float>((size_t)ch * batch * A.ld);
    A.pr = cv.take<float>((size_t)ch * batch * A.ld);
    if (p->phased) {
        A.in_c = G.c_i;
        A.in_s = G.sn_i;
    }
    LX_TRY(lx::scan_launch(A, s), "scan over the input side");
    lx::EvalGradArgs E;
    E.channels = ch;
    E.n_out = G.no;
    E.n_in = G.ni;
    E.batch = batch;
    E.ld = A.ld;
    E.inv_t = (float)p->inv_t;
    E.anchor_scale = p->temperature > 0.0 ? (float)(-1.0 / p->temperature) : 0.f;
    E.out_anchor = G.anchor_o;
    if (p->phased) {
        E.out_cos = G.c_o0;
        E.out_sin = G.s_o0;
    }
    E.s_in = G.s_i;
    E.pl = A.pl;
    E.pr = A.pr;
    E.w = W;
    E.y = y;
    E.d_anchor = d_anchor;
    E.d_phase = d_phase;
    E.lds_bytes = p->lds_bytes;
    LX_TRY(lx::eval_grad_launch(E, s), "evaluate gradients");
    return LAPLEX_OK;
}

}  // namespace

extern "C" {

laplex_status laplex_backward(laplex_plan p, const float* x, const float* g, int64_t batch, int transpose,
                              float* dx, float* da, float* db, float* dphi, float* dpsi, void* stream)
{
    if (!p) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "plan is NULL");
    if (!g) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "g is NULL");
    if (batch < 1) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "batch must be >= 1");
    if (transpose != 0 && transpose != 1) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "transpose must be 0 or 1");
    // x == NULL: the input kept by laplex_plan_create_apply (y = K x, so transpose 0)
    const bool use_kept = x == nullptr;
    if (use_kept && !p->kept_x) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "x is NULL and the plan keeps no input");
    if (use_kept && (transpose != 0 || batch != p->kept_batch))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "the kept input is for transpose = 0 and its own batch");
    const bool kept_by_rank = use_kept && p->kept_by_rank;
    if (use_kept && !kept_by_rank) x = p->kept_x;
    if (p->sym && db) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "symmetric plan: the gradient of b = a is in da");
    if (!p->phased && (dphi || dpsi)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "unphased plan has no phase gradients");
    const int64_t len_in = transpose ? p->n : p->k;
    const int64_t len_out = transpose ? p->k : p->n;
    if (batch > (int64_t)1 << 40 || (double)batch * (double)(len_in > len_out ? len_in : len_out) > 4.0e18 / 4)
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "batch too large");
    struct Range {
        const void* p;
        size_t bytes;
    };
    const Range outs[5] = {{dx, (size_t)(batch * len_in) * 4}, {da, (size_t)p->n * 4}, {db, (size_t)p->k * 4},
                           {dphi, (size_t)p->n * 4}, {dpsi, (size_t)p->k * 4}};
    const Range ins[2] = {{x, (size_t)(batch * len_in) * 4}, {g, (size_t)(batch * len_out) * 4}};
    for (int i = 0; i < 5; ++i) {
        if (!outs[i].p) continue;
        for (int j = 0; j < 2; ++j)
            if (ins[j].p && ranges_overlap(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes))
                return fail(LAPLEX_ERR_INVALID_ARGUMENT, "an output overlaps x or g");
        for (int j = i + 1; j < 5; ++j)
            if (outs[j].p && ranges_overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes))
                return fail(LAPLEX_ERR_INVALID_ARGUMENT, "two outputs overlap");
    }
    if (!dx && !da && !db && !dphi && !dpsi) return LAPLEX_OK;
    DeviceGuard guard(p->device);
    hipStream_t s = (hipStream_t)stream;
    note_stream(p, s);
    const int ch = p->phased ? 2 : 1;
    // row side u, column side w of F = sum <u, K w>
    const float* u = transpose ? x : g;
    const float* w = transpose ? g : x;
    const float anchor_scale = p->temperature > 0.0 ? (float)(-1.0 / p->temperature) : 0.f;

    if (p->sym) {
        const int64_t n = p->n;
        const bool replay = kept_by_rank || n >= replay_min();
        if (!replay) LX_TRY(ensure_perm(p, 0, s), "permutation");
        const int64_t ld = pad64(n);
        const int64_t tiles = (n + lx::kScanTile - 1) / lx::kScanTile;
        const int64_t groups = (tiles + lx::kCarryGroup - 1) / lx::kCarryGroup;
        const int64_t rows = 4 * (int64_t)ch * batch;
        const int64_t nout = (dx ? batch : 0) + (da ? 1 : 0) + (dphi ? 1 : 0) + (dpsi ? 1 : 0);
        const int64_t tmp_rows = replay ? (2 * batch > nout ? 2 * batch : nout) : batch;
        const size_t need = align256((size_t)rows * tiles * 4 * 8) + align256((size_t)rows * groups * 4 * 8) +
                            align256((size_t)rows * tiles * 2 * 8) + 2 * align256((size_t)tmp_rows * ld * 4);
        LX_TRY(ensure_ws(p, need, s), "workspace");
        Carve cv(p->ws);
        lx::GradSymArgs A;
        A.channels = ch;
        A.n = n;
        A.tiles = tiles;
        A.batch = batch;
        A.ld = ld;
        A.out_ld = ld;
        A.inv_t = p->inv_t;
        A.anchor_scale = anchor_scale;
        A.dx_half = transpose ? 0 : 1;
        A.s = p->sa;
        A.perm = p->pa;
        if (p->phased) {
            A.cphi = p->cphi;
            A.sphi = p->sphi;
            A.cpsi = p->cpsi;
            A.spsi = p->spsi;
        }
        A.agg = cv.take<double>((size_t)rows * tiles * 4);
        A.gagg = cv.take<double>((size_t)rows * groups * 4);
        A.carry = cv.take<double>((size_t)rows * tiles * 2);
        float* t1 = cv.take<float>((size_t)tmp_rows * ld);
        float* t2 = cv.take<float>((size_t)tmp_rows * ld);
        if (!replay) {
            A.random = true;
            A.u = u;
            A.w = w;
            A.us = t1;
            A.ws = t2;
            A.dx = dx;
            A.da = da;
            A.dphi = dphi;
            A.dpsi = dpsi;
            LX_TRY(lx::grad_sym_launch(A, s), "symmetric gradient");
            return LAPLEX_OK;
        }
        // u, w -> sorted order (rows [0, B) and [B, 2B)), gradient by rank into
        // t1, then the wanted rows back to original order.
        const lx::SortRecords& R = p->ra;
        A.random = false;
        if (kept_by_rank) {
            // w = x is already by rank: only u travels
            LX_TRY(lx::replay_launch(R, 0, true, u, n, t1, ld, batch, s), "replay");
            LX_TRY(lx::replay_launch(R, 1, true, t1, ld, t2, ld, batch, s), "replay");
            LX_TRY(lx::replay_launch(R, 2, true, t2, ld, t1, ld, batch, s), "replay");
            LX_TRY(lx::replay_launch(R, 3, true, t1, ld, t2, ld, batch, s), "replay");
            A.us = t2;
            A.ws = p->kept_x;
        } else {
            LX_TRY(lx::replay_launch(R, 0, true, u, n, t1, ld, batch, s), "replay");
            LX_TRY(lx::replay_launch(R, 0, true, w, n, t1 + batch * ld, ld, batch, s), "replay");
            LX_TRY(lx::replay_launch(R, 1, true, t1, ld, t2, ld, 2 * batch, s), "replay");
            LX_TRY(lx::replay_launch(R, 2, true, t2, ld, t1, ld, 2 * batch, s), "replay");
            LX_TRY(lx::replay_launch(R, 3, true, t1, ld, t2, ld, 2 * batch, s), "replay");
            A.us = t2;
            A.ws = t2 + batch * ld;
        }
        int64_t row = 0;
        float* user[4] = {dx, da, dphi, dpsi};
        int64_t first[4], count[4];
        for (int o = 0; o < 4; ++o) {
            count[o] = user[o] ? (o == 0 ? batch : 1) : 0;
            first[o] = row;
            row += count[o];
        }
        A.dx = dx ? t1 + first[0] * ld : nullptr;
        A.da = da ? t1 + first[1] * ld : nullptr;
        A.dphi = dphi ? t1 + first[2] * ld : nullptr;
        A.dpsi = dpsi ? t1 + first[3] * ld : nullptr;
        LX_TRY(lx::grad_sym_launch(A, s), "symmetric gradient");
        LX_TRY(lx::replay_launch(R, 3, false, t1, ld, t2, ld, nout, s), "replay");
        LX_TRY(lx::replay_launch(R, 2, false, t2, ld, t1, ld, nout, s), "replay");
        LX_TRY(lx::replay_launch(R, 1, false, t1, ld, t2, ld, nout, s), "replay");
        for (int o = 0; o < 4; ++o)
            if (count[o])
                LX_TRY(lx::replay_launch(R, 0, false, t2 + first[o] * ld, ld, user[o], n, count[o], s), "replay");
        return LAPLEX_OK;
    }

    // General plan: outputs on a from the tables of b, outputs on b from those of a.
    LX_TRY(ensure_perm(p, 0, s), "permutation of a");
    LX_TRY(ensure_perm(p, 1, s), "permutation of b");
    GradSide on_a{p->n, p->k, p->sb, p->pb, p->cpsi, p->spsi, p->a0, p->cphi0, p->sphi0,
                  p->sa, p->pa, p->b0, p->cpsi0, p->spsi0};
    GradSide on_b{p->k, p->n, p->sa, p->pa, p->cphi, p->sphi, p->b0, p->cpsi0, p->spsi0,
                  p->sb, p->pb, p->a0, p->cphi0, p->sphi0};
    laplex_status st = grad_general_side(p, on_a, w, u, batch, transpose ? dx : nullptr, da, dphi, s);
    if (st != LAPLEX_OK) return st;
    return grad_general_side(p, on_b, u, w, batch, transpose ? nullptr : dx, db, dpsi, s);
}

laplex_status laplex_gram(laplex_plan p, const float* D, float* M, void* stream)
{
    if (!p) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "plan is NULL");
    if (!D || !M) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "D or M is NULL");
    if ((double)p->n * (double)p->n > (double)((int64_t)1 << 40))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "n * n too large for a dense Gram matrix");
    if (ranges_overlap(D, (size_t)p->k * 4, M, (size_t)(p->n * p->n) * 4))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "D and M overlap");
    DeviceGuard g(p->device);
    hipStream_t s = (hipStream_t)stream;
    note_stream(p, s);
    LX_TRY(ensure_perm(p, 0, s), "permutation of a");
    LX_TRY(ensure_perm(p, 1, s), "permutation of b");
    if (!p->gbound) {
        void* gb = nullptr;
        LX_TRY(plan_alloc(p, &gb, (size_t)(p->n + 2) * 4, s), "alloc gram bounds");
        LX_TRY(lx::gram_bounds_launch(p->sa, p->n, p->sb, p->k, (uint32_t*)gb, s), "gram bounds");
        p->gbound = (uint32_t*)gb;
    }
    if (!p->grank) {
        void* gr = nullptr;
        LX_TRY(plan_alloc(p, &gr, (size_t)p->n * 4, s), "alloc gram ranks");
        LX_TRY(lx::gram_ranks_launch(p->pa, p->n, (uint32_t*)gr, s), "gram ranks");
        p->grank = (uint32_t*)gr;
    }
    LX_TRY(ensure_ws(p, lx::gram_scratch_bytes(p->n, p->k, p->phased ? 3 : 1), s), "workspace");
    lx::GramArgs G;
    G.n = p->n;
    G.k = p->k;
    G.inv_t = p->inv_t;
    G.sa = p->sa;
    G.pa = p->pa;
    G.sb = p->sb;
    G.pb = p->pb;
    G.D = D;
    G.bound = p->gbound;
    G.rank_a = p->grank;
    if (p->phased) {
        G.cphi_r = p->cphi;
        G.sphi_r = p->sphi;
        G.cpsi_r = p->cpsi;
        G.spsi_r = p->spsi;
    }
    if (!p->gslice_off) {
        void *off = nullptr, *src = nullptr, *bv = nullptr, *cv = nullptr, *sv = nullptr;
        LX_TRY(plan_alloc(p, &off, ((size_t)lx::kGramSlices * (p->n + 1) + 1) * 4, s), "alloc gram slices");
        LX_TRY(plan_alloc(p, &src, (size_t)p->k * 4, s), "alloc gram slices");
        LX_TRY(plan_alloc(p, &bv, (size_t)p->k * 4, s), "alloc gram slices");
        if (p->phased) {
            LX_TRY(plan_alloc(p, &cv, (size_t)p->k * 4, s), "alloc gram slices");
            LX_TRY(plan_alloc(p, &sv, (size_t)p->k * 4, s), "alloc gram slices");
        }
        LX_TRY(lx::gram_slices_launch(G, (uint32_t*)off, (uint32_t*)src, (float*)bv, (float*)cv, (float*)sv, s),
               "gram slices");
        p->gslice_off = (uint32_t*)off;
        p->gslice_src = (uint32_t*)src;
        p->gslice_b = (float*)bv;
        p->gslice_c = (float*)cv;
        p->gslice_s = (float*)sv;
    }
    G.slice_off = p->gslice_off;
    G.slice_src = p->gslice_src;
    G.slice_b = p->gslice_b;
    G.slice_c = p->gslice_c;
    G.slice_s = p->gslice_s;
    G.stats = (double*)p->ws;
    G.M = M;
    LX_TRY(lx::gram_launch(G, s), "gram");
    return LAPLEX_OK;
}

laplex_status laplex_profile_enable(int on)
{
    g_prof_on = on != 0;
    return LAPLEX_OK;
}

laplex_status laplex_profile_only(const char* label)
{
    g_prof_only = label ? label : "";
    return LAPLEX_OK;
}

laplex_status laplex_profile_reset(void)
{
    laplex_profile_collect();
    g_prof.clear();
    return LAPLEX_OK;
}

laplex_status laplex_profile_collect(void)
{
    laplex_status st = LAPLEX_OK;
    for (const Pending& q : g_pending) {
        float ms = 0.f;
        if (hipEventSynchronize(q.b) == hipSuccess && hipEventElapsedTime(&ms, q.a, q.b) == hipSuccess) {
            bool found = false;
            for (ProfEntry& e : g_prof)
                if (std::strcmp(e.name, q.name) == 0) {
                    e.launches += 1;
                    e.total_ms += ms;
                    found = true;
                    break;
                }
            if (!found) g_prof.push_back(ProfEntry{q.name, 1, (double)ms});
        } else {
            (void)hipGetLastError();
            st = fail(LAPLEX_ERR_DEVICE, "profiling event failed");
        }
        g_event_pool.push_back(q.a);
        g_event_pool.push_back(q.b);
    }
    g_pending.clear();
    return st;
}

laplex_status laplex_profile_entry(int i, const char** name, int64_t* launches, double* total_ms)
{
    if (i < 0 || i >= (int)g_prof.size()) return LAPLEX_ERR_INVALID_ARGUMENT;
    if (name) *name = g_prof[i].name;
    if (launches) *launches = g_prof[i].launches;
    if (total_ms) *total_ms = g_prof[i].total_ms;
    return LAPLEX_OK;
}

}  // extern "C"

// ------------------------------------------- token routing and recurrence
//
// Stateless calls: every array and all scratch are the caller's, so nothing
// here allocates, waits or records an event.

namespace {

struct Rows {  // an array of rows; width 0: absent
    const void* p;
    int64_t rows, ld, width;
    size_t size;
};

// Whether two arrays of rows share a byte.  Rows of one pitch may interleave
// (parts of one wider row).
bool rows_overlap(const Rows& a, const Rows& b)
{
    if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || a.width < 1 || b.width < 1) return false;
    const size_t sa = (size_t)a.ld * a.size, sb = (size_t)b.ld * b.size;
    const size_t wa = (size_t)a.width * a.size, wb = (size_t)b.width * b.size;
    if (!ranges_overlap(a.p, (size_t)(a.rows - 1) * sa + wa, b.p, (size_t)(b.rows - 1) * sb + wb)) return false;
    if (sa != sb || a.rows < 2 || b.rows < 2) return true;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    const size_t d = y >= x ? (size_t)(y - x) % sa : (sa - (size_t)(x - y) % sa) % sa;  // b's column in a's rows
    return d < wa || d + wb > sa;
}

const char* check_outputs(const Rows* outs, int n_out, const Rows* ins, int n_in)
{
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (rows_overlap(outs[i], ins[j])) return "an output overlaps an input";
        for (int j = i + 1; j < n_out; ++j)
            if (rows_overlap(outs[i], outs[j])) return "two outputs overlap";
    }
    return nullptr;
}

// Values of one array stay below 2^46: byte offsets stay far inside 63 bits.
bool rows_ok(const Rows& r)
{
    return !r.p || (r.ld >= r.width && r.ld <= (int64_t)1 << 40 && (double)r.rows * (double)r.ld < 7.0e13 &&
                    (uintptr_t)r.p % r.size == 0);
}

size_t dtype_size(laplex_dtype t) { return t == LAPLEX_F32 ? 4 : 2; }
bool dtype_ok(laplex_dtype t) { return t == LAPLEX_F32 || t == LAPLEX_BF16 || t == LAPLEX_F16; }

bool route_sizes_ok(int64_t tokens, int64_t slots)
{
    return tokens >= 0 && slots >= 1 && slots <= kMaxLen && tokens <= kMaxLen / slots;
}

bool recur_sizes_ok(int64_t n, int64_t width, int64_t heads)
{
    return n >= 0 && n <= 0x7FFFFFFF && width >= 1 && width <= (int64_t)1 << 24 && heads >= 1 && heads <= width &&
           width % heads == 0;
}

int64_t recur_tiles(int64_t n) { return (n + lx::kRecurTile - 1) / lx::kRecurTile; }
int64_t recur_cols(int64_t width) { return (width + lx::kRecurCols - 1) / lx::kRecurCols; }

// Fills the parts both directions share; a message if an argument is bad.
const char* recur_common(lx::RecurArgs& A, int64_t n, int64_t seqs, const int32_t* offsets, int64_t width,
                         int64_t heads, laplex_dtype type, laplex_dtype gate_type, const void* x, int64_t ldx,
                         const void* g, int64_t ldg, const float* h0)
{
    if (!recur_sizes_ok(n, width, heads)) return "bad sizes: 0 <= n < 2^31, 1 <= width <= 2^24, heads divides width";
    if (seqs < 1 || seqs > kMaxLen) return "seqs must be in [1, 2^30]";
    if (!offsets && n % seqs) return "without offsets n must be a multiple of seqs";
    if (!dtype_ok(type) || (gate_type != type && gate_type != LAPLEX_F32)) return "bad type or gate_type";
    if (n > 0 && (!x || !g)) return "x or g is NULL";
    const int64_t tiles = recur_tiles(n), cols = recur_cols(width);
    if (n > ((int64_t)1 << 38) / width) return "n * width must be at most 2^38";
    A.n = n;
    A.seqs = seqs;
    A.seq_len = offsets ? 0 : n / seqs;
    A.offsets = offsets;
    A.width = (int)width;
    A.heads = (int)heads;
    A.per = (int)(width / heads);
    // An array as large as the last-level cache (256 MB) is out of it again
    // before anyone else reads it.  Past the caches against through them, us:
    //   forward, then an operator that reads y, and backward, 4096 channels
    //              bf16 own decays      bf16 shared          float32 own          float32 shared
    //    64 MiB     74/ 70   84/ 91      64/ 59   68/ 68      72/ 67   81/ 87      58/ 52   55/ 53
    //   128 MiB    125/140  145/155     108/112  110/123     123/139  143/149     100/109   92/100
    //   256 MiB    234/247  262/284     201/207  190/209     234/251  277/276     189/200  162/173
    //   512 MiB    447/469  490/532     379/393  359/379     452/474  550/515     370/382  300/323
    // It would gain from 128 MiB on (with nothing else in the cache), and
    // loses up to 7 % of one form, the float32 backward with own decays.
    A.stream = (double)n * (double)width * (double)dtype_size(type) >= 268435456.0;
    A.tiles = tiles;
    A.cols = (int)cols;
    A.x = x;
    A.ldx = lx::recur_pitch(n, width, ldx);
    A.g = g;
    A.ldg = lx::recur_pitch(n, heads, ldg);
    A.h0 = h0;
    return nullptr;
}

// Scratch of a pass: tickets, marks, maps, states; none for a single row tile.
size_t recur_ticket_bytes(int64_t width) { return align256((size_t)recur_cols(width) * lx::kRecurTicketPitch * 4); }
size_t recur_mark_bytes(int64_t n) { return align256((size_t)recur_tiles(n) * 4); }
size_t recur_map_bytes(int64_t n, int64_t width)
{
    const int64_t t = recur_tiles(n);
    return t > 1 ? align256((size_t)((t - 1) * recur_cols(width) * lx::kRecurCols) * 8) : 0;
}
size_t recur_pass_bytes(int64_t n, int64_t width)
{
    const size_t m = recur_map_bytes(n, width);
    return m ? recur_ticket_bytes(width) + recur_mark_bytes(n) + m + align256(m / 2) : 0;
}
void recur_scratch(lx::RecurArgs& A, void* ws)
{
    char* p = (char*)ws;
    A.tickets = (uint32_t*)p;
    p += recur_ticket_bytes(A.width);
    A.marks = (int32_t*)p;
    p += recur_mark_bytes(A.n);
    A.maps = (uint64_t*)p;
    A.states = (uint32_t*)(p + recur_map_bytes(A.n, A.width));
    A.part = (float*)((char*)ws + recur_pass_bytes(A.n, A.width));
}

}  // namespace

extern "C" {

int64_t laplex_route_workspace(int64_t tokens, int64_t slots, int64_t n_experts)
{
    if (!route_sizes_ok(tokens, slots) || n_experts < 1 || n_experts > lx::kRouteMaxExperts) return -1;
    const int64_t tiles = (tokens * slots + lx::kRouteTile - 1) / lx::kRouteTile;
    return tokens * slots > lx::kRouteSingle ? (tiles + 1) * n_experts * 4 : 0;
}

laplex_status laplex_route(const void* experts, int wide, int64_t tokens, int64_t slots, int64_t n_experts,
                           int32_t* order, int32_t* place, int32_t* offsets, void* ws, int64_t ws_bytes,
                           void* stream)
{
    const int64_t need = laplex_route_workspace(tokens, slots, n_experts);
    if (need < 0)
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "tokens * slots must be at most 2^30 and n_experts in [1, 4096]");
    if (wide != 0 && wide != 1) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "wide must be 0 or 1");
    const int64_t n = tokens * slots;
    if (!offsets || (n > 0 && (!experts || !order || !place)))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "experts, order, place or offsets is NULL");
    if (need > 0 && (!ws || (uintptr_t)ws % 16 || ws_bytes < need))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "ws is NULL, misaligned or smaller than laplex_route_workspace");
    const Rows outs[4] = {{order, 1, n, n, 4}, {place, 1, n, n, 4}, {offsets, 1, n_experts + 1, n_experts + 1, 4},
                          {need > 0 ? ws : nullptr, 1, need, need, 1}};
    const Rows in = {experts, 1, n, n, wide ? 8u : 4u};
    if (!rows_ok(outs[0]) || !rows_ok(outs[1]) || !rows_ok(outs[2]) || !rows_ok(in))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "a misaligned array");
    if (const char* m = check_outputs(outs, 4, &in, 1)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, m);
    const laplex_status st = check_device();
    if (st != LAPLEX_OK) return st;
    lx::RouteArgs A;
    A.ids = experts;
    A.wide = wide;
    A.n = n;
    A.tiles = (n + lx::kRouteTile - 1) / lx::kRouteTile;
    A.experts = (int)n_experts;
    A.order = order;
    A.place = place;
    A.offsets = offsets;
    A.hist = (uint32_t*)ws;
    A.total = need > 0 ? (uint32_t*)ws + A.tiles * n_experts : nullptr;
    LX_TRY(lx::route_launch(A, (hipStream_t)stream), "route");
    return LAPLEX_OK;
}

laplex_status laplex_dispatch(int64_t tokens, int64_t slots, int64_t n_experts, const int32_t* place,
                              const int32_t* offsets, laplex_dtype type, int64_t width, const void* x, int64_t ldx,
                              void* xs, int64_t ldxs, void* stream)
{
    if (!route_sizes_ok(tokens, slots) || n_experts < 1 || n_experts > lx::kRouteMaxExperts || width < 1 ||
        width > (int64_t)1 << 24 || !dtype_ok(type))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "bad sizes or type");
    if (tokens == 0) return LAPLEX_OK;
    if (!place || !offsets || !x || !xs) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "place, offsets, x or xs is NULL");
    const size_t e = dtype_size(type);
    const Rows out = {xs, tokens * slots, ldxs, width, e};
    const Rows ins[3] = {{x, tokens, ldx, width, e}, {place, tokens, slots, slots, 4},
                         {offsets, 1, n_experts + 1, n_experts + 1, 4}};
    if (!rows_ok(out) || !rows_ok(ins[0])) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "a bad row pitch or alignment");
    if (const char* m = check_outputs(&out, 1, ins, 3)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, m);
    const laplex_status st = check_device();
    if (st != LAPLEX_OK) return st;
    lx::MoveArgs A;
    A.tokens = tokens;
    A.slots = slots;
    A.width = width;
    A.experts = (int)n_experts;
    A.place = place;
    A.offsets = offsets;
    A.in = x;
    A.ld_in = ldx;
    A.out = xs;
    A.ld_out = ldxs;
    LX_TRY(lx::move_rows_launch(lx::kMoveDispatch, (int)type, A, (hipStream_t)stream), "dispatch");
    return LAPLEX_OK;
}

laplex_status laplex_combine(int64_t tokens, int64_t slots, const int32_t* place, laplex_dtype type, int64_t width,
                             const void* ys, int64_t ldys, const float* weights, void* y, int64_t ldy,
                             void* stream)
{
    if (!route_sizes_ok(tokens, slots) || width < 1 || width > (int64_t)1 << 24 || !dtype_ok(type))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "bad sizes or type");
    if (tokens == 0) return LAPLEX_OK;
    if (!place || !ys || !y) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "place, ys or y is NULL");
    const size_t e = dtype_size(type);
    const Rows out = {y, tokens, ldy, width, e};
    const Rows ins[3] = {{ys, tokens * slots, ldys, width, e}, {place, tokens, slots, slots, 4},
                         {weights, tokens, slots, slots, 4}};
    if (!rows_ok(out) || !rows_ok(ins[0])) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "a bad row pitch or alignment");
    if (const char* m = check_outputs(&out, 1, ins, 3)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, m);
    const laplex_status st = check_device();
    if (st != LAPLEX_OK) return st;
    lx::MoveArgs A;
    A.tokens = tokens;
    A.slots = slots;
    A.width = width;
    A.place = place;
    A.weights = weights;
    A.in = ys;
    A.ld_in = ldys;
    A.out = y;
    A.ld_out = ldy;
    LX_TRY(lx::move_rows_launch(lx::kMoveCombine, (int)type, A, (hipStream_t)stream), "combine");
    return LAPLEX_OK;
}

laplex_status laplex_combine_backward(int64_t tokens, int64_t slots, int64_t n_experts, const int32_t* place,
                                      const int32_t* offsets, laplex_dtype type, int64_t width, const void* dy,
                                      int64_t lddy, const void* ys, int64_t ldys, const float* weights, void* dys,
                                      int64_t lddys, float* dweights, void* stream)
{
    if (!route_sizes_ok(tokens, slots) || n_experts < 1 || n_experts > lx::kRouteMaxExperts || width < 1 ||
        width > (int64_t)1 << 24 || !dtype_ok(type))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "bad sizes or type");
    if (tokens == 0 || (!dys && !dweights)) return LAPLEX_OK;
    if (!place || !dy || (dys && (!weights || !offsets)) || (dweights && !ys))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "place, dy, or what dys or dweights needs is NULL");
    const size_t e = dtype_size(type);
    const Rows outs[2] = {{dys, tokens * slots, lddys, width, e}, {dweights, tokens, slots, slots, 4}};
    const Rows ins[5] = {{dy, tokens, lddy, width, e}, {dweights ? ys : nullptr, tokens * slots, ldys, width, e},
                         {place, tokens, slots, slots, 4}, {weights, tokens, slots, slots, 4},
                         {offsets, 1, n_experts + 1, n_experts + 1, 4}};
    if (!rows_ok(outs[0]) || !rows_ok(ins[0]) || !rows_ok(ins[1]))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "a bad row pitch or alignment");
    if (const char* m = check_outputs(outs, 2, ins, 5)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, m);
    const laplex_status st = check_device();
    if (st != LAPLEX_OK) return st;
    lx::MoveArgs A;
    A.tokens = tokens;
    A.slots = slots;
    A.width = width;
    A.experts = (int)n_experts;
    A.place = place;
    A.offsets = offsets;
    A.weights = weights;
    A.in = dweights ? ys : nullptr;
    A.ld_in = ldys;
    A.dy = dy;
    A.ld_dy = lddy;
    A.out = dys;
    A.ld_out = lddys;
    A.dw = dweights;
    LX_TRY(lx::move_rows_launch(lx::kMoveCombineGrad, (int)type, A, (hipStream_t)stream), "combine backward");
    return LAPLEX_OK;
}

int64_t laplex_recur_states(int64_t n, int64_t width)
{
    if (!recur_sizes_ok(n, width, 1)) return -1;
    const int64_t t = recur_tiles(n);
    return t > 1 ? (t - 1) * recur_cols(width) * lx::kRecurCols : 0;
}

int64_t laplex_recur_workspace(int64_t n, int64_t width, int64_t heads, int backward)
{
    if (!recur_sizes_ok(n, width, heads) || (backward != 0 && backward != 1)) return -1;
    size_t b = recur_pass_bytes(n, width);
    if (backward && heads < width && !lx::recur_heads_inside((int)width, (int)(width / heads)))
        b += align256((size_t)n * (size_t)(recur_cols(width) + heads) * 4);
    return (int64_t)b;
}

laplex_status laplex_recur(int64_t n, int64_t seqs, const int32_t* offsets, int64_t width, int64_t heads,
                           laplex_dtype type, laplex_dtype gate_type, const void* x, int64_t ldx, const void* g,
                           int64_t ldg, const float* h0, void* y, int64_t ldy, float* final, float* states,
                           void* ws, int64_t ws_bytes, void* stream)
{
    lx::RecurArgs A;
    if (const char* m = recur_common(A, n, seqs, offsets, width, heads, type, gate_type, x, ldx, g, ldg, h0))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, m);
    if (n > 0 && !y) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "y is NULL");
    const int64_t need = laplex_recur_workspace(n, width, heads, 0);
    if (need > 0 && (!ws || (uintptr_t)ws % 16 || ws_bytes < need))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "ws is NULL, misaligned or smaller than laplex_recur_workspace");
    const size_t e = dtype_size(type), eg = dtype_size(gate_type);
    const int64_t ns = laplex_recur_states(n, width);
    if (ns > 0 && (uintptr_t)states % 16) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "states must be 16-byte aligned");
    const Rows outs[4] = {{y, n, ldy, width, e}, {final, seqs, width, width, 4},
                          {ns > 0 ? states : nullptr, 1, ns, ns, 4}, {need > 0 ? ws : nullptr, 1, need, need, 1}};
    const Rows ins[4] = {{x, n, ldx, width, e}, {g, n, ldg, heads, eg}, {h0, seqs, width, width, 4},
                         {offsets, 1, seqs + 1, seqs + 1, 4}};
    for (const Rows& r : {outs[0], outs[1], ins[0], ins[1], ins[2]})
        if (!rows_ok(r) || (r.rows > 1 && r.ld > lx::kRecurMaxPitch))
            return fail(LAPLEX_ERR_INVALID_ARGUMENT, "a bad row pitch or alignment");
    if (const char* m = check_outputs(outs, 4, ins, 4)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, m);
    const laplex_status st = check_device();
    if (st != LAPLEX_OK) return st;
    hipStream_t s = (hipStream_t)stream;
    A.y = y;
    A.ldy = lx::recur_pitch(n, width, ldy);
    A.final = final;
    recur_scratch(A, ws);
    if (states) A.states = (uint32_t*)states;
    LX_TRY(lx::recur_launch(A, (int)type, gate_type == LAPLEX_F32 ? 0 : (int)type, s), "recurrence");
    return LAPLEX_OK;
}

laplex_status laplex_recur_backward(int64_t n, int64_t seqs, const int32_t* offsets, int64_t width, int64_t heads,
                                    laplex_dtype type, laplex_dtype gate_type, const void* x, int64_t ldx,
                                    const void* g, int64_t ldg, const float* h0, const float* states,
                                    const void* dy, int64_t lddy, const float* dfinal, void* dx, int64_t lddx,
                                    void* dg, int64_t lddg, float* dh0, void* ws, int64_t ws_bytes, void* stream)
{
    lx::RecurArgs A;
    if (const char* m = recur_common(A, n, seqs, offsets, width, heads, type, gate_type, x, ldx, g, ldg, h0))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, m);
    if (!dx && !dg && !dh0) return LAPLEX_OK;
    if (n > 0 && !dy) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "dy is NULL");
    const int64_t ns = laplex_recur_states(n, width);
    if (ns > 0 && !states) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "states is NULL");
    const int64_t need = laplex_recur_workspace(n, width, heads, 1);
    if (need > 0 && (!ws || (uintptr_t)ws % 16 || ws_bytes < need))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "ws is NULL, misaligned or smaller than laplex_recur_workspace");
    const size_t e = dtype_size(type), eg = dtype_size(gate_type);
    const Rows outs[4] = {{dx, n, lddx, width, e}, {dg, n, lddg, heads, eg}, {dh0, seqs, width, width, 4},
                          {need > 0 ? ws : nullptr, 1, need, need, 1}};
    const Rows ins[7] = {{x, n, ldx, width, e}, {g, n, ldg, heads, eg}, {h0, seqs, width, width, 4},
                         {offsets, 1, seqs + 1, seqs + 1, 4}, {dy, n, lddy, width, e},
                         {dfinal, seqs, width, width, 4}, {ns > 0 ? states : nullptr, 1, ns, ns, 4}};
    for (const Rows& r : {outs[0], outs[1], outs[2], ins[0], ins[1], ins[2], ins[4], ins[5], ins[6]})
        if (!rows_ok(r) || (r.rows > 1 && r.ld > lx::kRecurMaxPitch))
            return fail(LAPLEX_ERR_INVALID_ARGUMENT, "a bad row pitch or alignment");
    if (const char* m = check_outputs(outs, 4, ins, 7)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, m);
    const laplex_status st = check_device();
    if (st != LAPLEX_OK) return st;
    hipStream_t s = (hipStream_t)stream;
    A.dy = dy;
    A.lddy = lx::recur_pitch(n, width, lddy);
    A.dfinal = dfinal;
    A.states_in = states;
    A.dx = dx;
    A.lddx = lx::recur_pitch(n, width, lddx);
    A.dg = dg;
    A.lddg = lx::recur_pitch(n, heads, lddg);
    A.dh0 = dh0;
    recur_scratch(A, ws);
    LX_TRY(lx::recur_grad_launch(A, (int)type, gate_type == LAPLEX_F32 ? 0 : (int)type, s), "recurrence backward");
    return LAPLEX_OK;
}

laplex_status laplex_recur_step(int64_t n, int64_t pool, const int32_t* slots, int64_t width, int64_t heads,
                                laplex_dtype type, laplex_dtype gate_type, const void* x, int64_t ldx,
                                const void* g, int64_t ldg, float* state, void* y, int64_t ldy, void* stream)
{
    if (!recur_sizes_ok(n, width, heads) || pool < 0 || pool > 0x7FFFFFFF)
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "bad sizes: 0 <= n, pool < 2^31, 1 <= width <= 2^24, heads divides width");
    if (!dtype_ok(type) || (gate_type != type && gate_type != LAPLEX_F32))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "bad type or gate_type");
    if (!slots && n > pool) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "without slots n must be at most pool");
    if (n == 0) return LAPLEX_OK;
    if (!x || !g || !y || (pool > 0 && !state)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "x, g, state or y is NULL");
    const size_t e = dtype_size(type), eg = dtype_size(gate_type);
    const Rows outs[2] = {{y, n, ldy, width, e}, {state, pool, width, width, 4}};
    const Rows ins[3] = {{x, n, ldx, width, e}, {g, n, ldg, heads, eg}, {slots, 1, n, n, 4}};
    for (const Rows& r : {outs[0], outs[1], ins[0], ins[1]})
        if (!rows_ok(r)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "a bad row pitch or alignment");
    if (const char* m = check_outputs(outs, 2, ins, 3)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, m);
    const laplex_status st = check_device();
    if (st != LAPLEX_OK) return st;
    lx::RecurStepArgs A;
    A.n = n;
    A.pool = pool;
    A.width = (int)width;
    A.heads = (int)heads;
    A.per = (int)(width / heads);
    A.x = x;
    A.g = g;
    A.y = y;
    A.ldx = ldx;
    A.ldg = ldg;
    A.ldy = ldy;
    A.slots = slots;
    A.state = state;
    LX_TRY(lx::recur_step_launch(A, (int)type, gate_type == LAPLEX_F32 ? 0 : (int)type, (hipStream_t)stream),
           "recurrence step");
    return LAPLEX_OK;
}

}  // extern "C"

// ---- experts' products and the gated matrix memory ----

namespace {

// Experts' matrices [experts][rows][cols]: everything between the first and
// the last value.
Rows matrices(const void* p, int64_t experts, int64_t rows, int64_t cols, int64_t ld, int64_t pitch, size_t size)
{
    const int64_t span = (experts - 1) * pitch + (rows - 1) * ld + cols;
    return Rows{p, 1, span, span, size};
}

bool matrices_ok(const void* p, int64_t experts, int64_t rows, int64_t cols, int64_t ld, int64_t pitch, size_t size)
{
    return ld >= cols && ld <= (int64_t)1 << 40 && pitch >= 0 && pitch <= (int64_t)1 << 46 &&
           (double)experts * (double)pitch + (double)rows * (double)ld < 7.0e13 && (uintptr_t)p % size == 0;
}

bool experts_sizes_ok(int64_t n, int64_t n_experts, int64_t in, int64_t out, laplex_dtype type, int transpose)
{
    return n >= 0 && n <= 0x7FFFFFFF && n_experts >= 1 && n_experts <= lx::kRouteMaxExperts && in >= 1 &&
           in <= (int64_t)1 << 24 && out >= 1 && out <= (int64_t)1 << 24 && dtype_ok(type) &&
           (transpose == 0 || transpose == 1);
}

constexpr const char* kBadExperts =
    "bad sizes, type or transpose: 0 <= n < 2^31, n_experts in [1, 4096], in and out in [1, 2^24]";

// Sizes of a pass of the matrix memory, the same for both directions.
constexpr int kAttendMaxHeads = 4096, kAttendMaxDim = 1024;
bool attend_sizes(lx::AttendArgs& A, int64_t n, int64_t seqs, int64_t heads, int64_t hq, int64_t hk, int64_t hv, int64_t dk,
                  int64_t dv, laplex_dtype type)
{
    if (n < 0 || n > 0x7FFFFFFF || seqs < 1 || seqs > (int64_t)1 << 24 || heads < 1 || heads > kAttendMaxHeads || dk < 1 || dk > kAttendMaxDim || dv < 1 ||
        dv > kAttendMaxDim || !dtype_ok(type))
        return false;
    for (int64_t h : {hq, hk, hv})
        if (h < 1 || h > heads || heads % h) return false;
    A.n = n;
    A.heads = (int)heads;
    A.hq = (int)hq;
    A.hk = (int)hk;
    A.hv = (int)hv;
    A.dk = (int)dk;
    A.dv = (int)dv;
    A.block_k = dk <= 64 ? 64 : 128;
    A.nkb = (int)((dk + A.block_k - 1) / A.block_k);
    A.nvb = (int)((dv + 63) / 64);
    A.dkp = A.nkb * A.block_k;
    A.dvp = A.nvb * 64;
    A.grad_block_k = type == LAPLEX_BF16 ? A.block_k : 64;
    A.loop = hq == hk ? (int)(heads / hq) : 1;
    A.segment = lx::attend_segment(n, seqs, heads * A.nkb * (A.nvb % 2 ? A.nvb : A.nvb / 2));
    // states of all slots between chunks stay below 2^46 bytes
    return (double)(n / lx::kAttendChunk + 1) * (double)heads * A.dkp * A.dvp < 1.7e13;
}

int64_t attend_slots(const lx::AttendArgs& A) { return A.n > A.segment ? A.n / A.segment : 0; }
size_t attend_slot_values(const lx::AttendArgs& A) { return (size_t)A.heads * A.dkp * A.dvp; }

// Lays out the scratch from `base` on; its size.
size_t attend_carve(lx::AttendArgs& A, char* base, bool backward, bool own_states)
{
    size_t off = 0;
    auto take = [&](size_t values) {
        float* p = values ? (float*)(base + off) : nullptr;
        off += align256(values * 4);
        return p;
    };
    const size_t slots = (size_t)attend_slots(A), one = attend_slot_values(A), n = (size_t)A.n;
    A.seg_decays = take(slots * A.heads);
    if (!backward) {
        if (own_states) A.seg_states = take(slots * one);
        A.part = take(A.nkb > 1 ? (size_t)A.nkb * n * A.heads * A.dv : 0);
        return off;
    }
    A.seg_grads = take(slots * one);
    A.chunk_states = take(n / lx::kAttendChunk * one);
    A.chunk_grads = take(n / lx::kAttendChunk * one);
    const size_t nkb = (size_t)lx::attend_grad_blocks(A);
    const size_t rq = A.heads / A.hq / A.loop, rk = A.heads / A.hk / A.loop, rv = A.heads / A.hv * nkb;
    A.part_q = take(rq > 1 ? rq * n * A.hq * A.dk : 0);
    A.part_k = take(rk > 1 ? rk * n * A.hk * A.dk : 0);
    A.part_v = take(rv > 1 ? rv * n * A.hv * A.dv : 0);
    A.part_g = take(nkb > 1 ? nkb * n * A.heads : 0);
    return off;
}

constexpr const char* kBadAttend =
    "bad sizes or type: 0 <= n < 2^31, seqs in [1, 2^24], heads in [1, 4096] and a multiple of each array's, dk and dv in [1, 1024]";

const char* attend_common(lx::AttendArgs& A, int64_t n, int64_t seqs, const int32_t* offsets, int64_t heads,
                          int64_t hq, int64_t hk, int64_t hv, int64_t dk, int64_t dv, laplex_dtype type,
                          laplex_dtype gate_type, float scale, const void* q, int64_t ldq, const void* k, int64_t ldk,
                          const void* v, int64_t ldv, const void* g, int64_t ldg, const float* h0)
{
    if (!attend_sizes(A, n, seqs, heads, hq, hk, hv, dk, dv, type)) return kBadAttend;
    if (!offsets && n % seqs) return "without offsets n must be a multiple of seqs";
    if (gate_type != type && gate_type != LAPLEX_F32) return "bad gate_type";
    if (n > 0 && (!q || !k || !v || !g)) return "q, k, v or g is NULL";
    if ((double)(n / lx::kAttendChunk + seqs + 2) * (double)heads * A.nkb * 2 * A.nvb > 1.3e11)
        return "too many sequences for so many heads";
    A.seqs = seqs;
    A.seq_len = offsets ? 0 : n / seqs;
    A.offsets = offsets;
    A.scale = scale;
    A.q = q;
    A.k = k;
    A.v = v;
    A.g = g;
    A.ldq = ldq;
    A.ldk = ldk;
    A.ldv = ldv;
    A.ldg = ldg;
    A.h0 = h0;
    return nullptr;
}

}  // namespace

extern "C" {

laplex_status laplex_experts(int64_t n, int64_t n_experts, const int32_t* offsets, int64_t in, int64_t out,
                             laplex_dtype type, int transpose, const void* x, int64_t ldx, const void* w, int64_t ldw,
                             int64_t pitch, void* y, int64_t ldy, void* stream)
{
    if (!experts_sizes_ok(n, n_experts, in, out, type, transpose)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, kBadExperts);
    if (n == 0) return LAPLEX_OK;
    if (!offsets || !x || !w || !y) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "offsets, x, w or y is NULL");
    const size_t e = dtype_size(type);
    const int64_t rw = transpose ? in : out, cw = transpose ? out : in;
    if (!matrices_ok(w, n_experts, rw, cw, ldw, pitch, e))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "a bad pitch or alignment of w");
    const Rows o = {y, n, ldy, out, e};
    const Rows ins[3] = {{x, n, ldx, in, e}, matrices(w, n_experts, rw, cw, ldw, pitch, e),
                         {offsets, 1, n_experts + 1, n_experts + 1, 4}};
    if (!rows_ok(o) || !rows_ok(ins[0]) || !rows_ok(ins[2]))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "a bad row pitch or alignment");
    if (const char* m = check_outputs(&o, 1, ins, 3)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, m);
    const laplex_status st = check_device();
    if (st != LAPLEX_OK) return st;
    lx::ExpertsArgs A;
    A.n = n;
    A.experts = n_experts;
    A.offsets = offsets;
    A.in = in;
    A.out = out;
    A.transpose = transpose;
    A.x = x;
    A.ldx = ldx;
    A.w = w;
    A.ldw = ldw;
    A.pitch_w = pitch;
    A.y = y;
    A.ldy = ldy;
    LX_TRY(lx::experts_launch(A, (int)type, (hipStream_t)stream), "experts");
    return LAPLEX_OK;
}

laplex_status laplex_experts_backward(int64_t n, int64_t n_experts, const int32_t* offsets, int64_t in, int64_t out,
                                      laplex_dtype type, int transpose, const void* x, int64_t ldx, const void* w,
                                      int64_t ldw, int64_t pitch, const void* dy, int64_t lddy, void* dx,
                                      int64_t lddx, void* dw, int64_t lddw, int64_t pitch_dw, void* stream)
{
    if (!experts_sizes_ok(n, n_experts, in, out, type, transpose)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, kBadExperts);
    if (!dx && !dw) return LAPLEX_OK;
    if (!offsets || (n > 0 && (!dy || (dw && !x) || (dx && !w))))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "offsets, dy, or what dx or dw needs is NULL");
    const size_t e = dtype_size(type);
    const int64_t rw = transpose ? in : out, cw = transpose ? out : in;
    if ((dx && n > 0 && !matrices_ok(w, n_experts, rw, cw, ldw, pitch, e)) ||
        (dw && (!matrices_ok(dw, n_experts, rw, cw, lddw, pitch_dw, e) ||
                (n_experts > 1 && pitch_dw < (rw - 1) * lddw + cw))))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "a bad pitch or alignment of w or dw");
    const Rows none = {nullptr, 0, 0, 0, 1};
    const Rows outs[2] = {n > 0 ? Rows{dx, n, lddx, in, e} : none,
                          dw ? matrices(dw, n_experts, rw, cw, lddw, pitch_dw, e) : none};
    const Rows ins[4] = {n > 0 ? Rows{dy, n, lddy, out, e} : none, dw && n > 0 ? Rows{x, n, ldx, in, e} : none,
                         dx && n > 0 ? matrices(w, n_experts, rw, cw, ldw, pitch, e) : none,
                         {offsets, 1, n_experts + 1, n_experts + 1, 4}};
    if (!rows_ok(outs[0]) || !rows_ok(ins[0]) || !rows_ok(ins[1]) || !rows_ok(ins[3]))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "a bad row pitch or alignment");
    if (const char* m = check_outputs(outs, 2, ins, 4)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, m);
    const laplex_status st = check_device();
    if (st != LAPLEX_OK) return st;
    lx::ExpertsArgs A;
    A.n = n;
    A.experts = n_experts;
    A.offsets = offsets;
    if (dx && n > 0) {  // the product with the other side's matrix
        A.in = out;
        A.out = in;
        A.transpose = !transpose;
        A.x = dy;
        A.ldx = lddy;
        A.w = w;
        A.ldw = ldw;
        A.pitch_w = pitch;
        A.y = dx;
        A.ldy = lddx;
        LX_TRY(lx::experts_launch(A, (int)type, (hipStream_t)stream), "experts backward");
    }
    if (dw) {  // its rows from dy, its columns from x; the other way round for transposed ones
        A.in = transpose ? out : in;
        A.out = transpose ? in : out;
        A.x = transpose ? dy : x;
        A.ldx = transpose ? lddy : ldx;
        A.y = const_cast<void*>(transpose ? x : dy);
        A.ldy = transpose ? ldx : lddy;
        A.dw = dw;
        A.ldw = lddw;
        A.pitch_w = pitch_dw;
        LX_TRY(lx::experts_grad_launch(A, (int)type, (hipStream_t)stream), "experts backward");
    }
    return LAPLEX_OK;
}

int64_t laplex_attend_states(int64_t n, int64_t seqs, int64_t heads, int64_t dk, int64_t dv)
{
    lx::AttendArgs A;
    if (!attend_sizes(A, n, seqs, heads, heads, heads, heads, dk, dv, LAPLEX_F32)) return -1;
    return attend_slots(A) * (int64_t)attend_slot_values(A);
}

int64_t laplex_attend_workspace(int64_t n, int64_t seqs, int64_t heads, int64_t query_heads, int64_t key_heads,
                                int64_t value_heads, int64_t dk, int64_t dv, laplex_dtype type, int backward)
{
    lx::AttendArgs A;
    if ((backward != 0 && backward != 1) ||
        !attend_sizes(A, n, seqs, heads, query_heads, key_heads, value_heads, dk, dv, type))
        return -1;
    return (int64_t)attend_carve(A, nullptr, backward, true);
}

laplex_status laplex_attend(int64_t n, int64_t seqs, const int32_t* offsets, int64_t heads, int64_t query_heads,
                            int64_t key_heads, int64_t value_heads, int64_t dk, int64_t dv, laplex_dtype type,
                            laplex_dtype gate_type, float scale, const void* q, int64_t ldq, const void* k,
                            int64_t ldk, const void* v, int64_t ldv, const void* g, int64_t ldg, const float* h0,
                            void* y, int64_t ldy, float* final, float* states, void* ws, int64_t ws_bytes,
                            void* stream)
{
    lx::AttendArgs A;
    if (const char* m = attend_common(A, n, seqs, offsets, heads, query_heads, key_heads, value_heads, dk, dv, type,
                                      gate_type, scale, q, ldq, k, ldk, v, ldv, g, ldg, h0))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, m);
    if (n > 0 && !y) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "y is NULL");
    const int64_t need =
        laplex_attend_workspace(n, seqs, heads, query_heads, key_heads, value_heads, dk, dv, type, 0);
    if (need > 0 && (!ws || (uintptr_t)ws % 16 || ws_bytes < need))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "ws is NULL, misaligned or smaller than laplex_attend_workspace");
    const size_t e = dtype_size(type), eg = dtype_size(gate_type);
    const int64_t ns = laplex_attend_states(n, seqs, heads, dk, dv), one = heads * dk * dv;
    if (ns > 0 && (uintptr_t)states % 16) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "states must be 16-byte aligned");
    const Rows outs[4] = {{y, n, ldy, heads * dv, e}, {final, seqs, one, one, 4},
                          {ns > 0 ? states : nullptr, 1, ns, ns, 4}, {need > 0 ? ws : nullptr, 1, need, need, 1}};
    const Rows ins[6] = {{q, n, ldq, query_heads * dk, e}, {k, n, ldk, key_heads * dk, e},
                         {v, n, ldv, value_heads * dv, e}, {g, n, ldg, heads, eg}, {h0, seqs, one, one, 4},
                         {offsets, 1, seqs + 1, seqs + 1, 4}};
    for (const Rows& r : {outs[0], outs[1], ins[0], ins[1], ins[2], ins[3], ins[4], ins[5]})
        if (!rows_ok(r)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "a bad row pitch or alignment");
    if (const char* m = check_outputs(outs, 4, ins, 6)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, m);
    const laplex_status st = check_device();
    if (st != LAPLEX_OK) return st;
    attend_carve(A, (char*)ws, false, true);
    if (states) A.seg_states = states;
    A.y = y;
    A.ldy = ldy;
    A.final = final;
    LX_TRY(lx::attend_launch(A, (int)type, gate_type == LAPLEX_F32 ? 0 : (int)type, (hipStream_t)stream), "attend");
    return LAPLEX_OK;
}

laplex_status laplex_attend_backward(int64_t n, int64_t seqs, const int32_t* offsets, int64_t heads,
                                     int64_t query_heads, int64_t key_heads, int64_t value_heads, int64_t dk,
                                     int64_t dv, laplex_dtype type, laplex_dtype gate_type, float scale,
                                     const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v,
                                     int64_t ldv, const void* g, int64_t ldg, const float* h0, const float* states,
                                     const void* dy, int64_t lddy, const float* dfinal, void* dq, int64_t lddq,
                                     void* dk_out, int64_t lddk, void* dv_out, int64_t lddv, void* dg, int64_t lddg,
                                     float* dh0, void* ws, int64_t ws_bytes, void* stream)
{
    lx::AttendArgs A;
    if (const char* m = attend_common(A, n, seqs, offsets, heads, query_heads, key_heads, value_heads, dk, dv, type,
                                      gate_type, scale, q, ldq, k, ldk, v, ldv, g, ldg, h0))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, m);
    if (!dq && !dk_out && !dv_out && !dg && !dh0) return LAPLEX_OK;
    if (n > 0 && !dy) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "dy is NULL");
    const int64_t ns = laplex_attend_states(n, seqs, heads, dk, dv), one = heads * dk * dv;
    if (ns > 0 && (!states || (uintptr_t)states % 16))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "states is NULL or misaligned");
    const int64_t need =
        laplex_attend_workspace(n, seqs, heads, query_heads, key_heads, value_heads, dk, dv, type, 1);
    if (need > 0 && (!ws || (uintptr_t)ws % 16 || ws_bytes < need))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "ws is NULL, misaligned or smaller than laplex_attend_workspace");
    const size_t e = dtype_size(type), eg = dtype_size(gate_type);
    const Rows outs[6] = {{dq, n, lddq, query_heads * dk, e}, {dk_out, n, lddk, key_heads * dk, e},
                          {dv_out, n, lddv, value_heads * dv, e}, {dg, n, lddg, heads, eg}, {dh0, seqs, one, one, 4},
                          {need > 0 ? ws : nullptr, 1, need, need, 1}};
    const Rows ins[9] = {{q, n, ldq, query_heads * dk, e}, {k, n, ldk, key_heads * dk, e},
                         {v, n, ldv, value_heads * dv, e}, {g, n, ldg, heads, eg}, {dy, n, lddy, heads * dv, e},
                         {h0, seqs, one, one, 4}, {dfinal, seqs, one, one, 4},
                         {ns > 0 ? states : nullptr, 1, ns, ns, 4}, {offsets, 1, seqs + 1, seqs + 1, 4}};
    for (int i = 0; i < 5; ++i)
        if (!rows_ok(outs[i])) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "a bad row pitch or alignment");
    for (const Rows& r : ins)
        if (!rows_ok(r)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "a bad row pitch or alignment");
    if (const char* m = check_outputs(outs, 6, ins, 9)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, m);
    const laplex_status st = check_device();
    if (st != LAPLEX_OK) return st;
    attend_carve(A, (char*)ws, true, false);
    A.seg_states = const_cast<float*>(states);  // read only
    A.dy = dy;
    A.lddy = lddy;
    A.dfinal = dfinal;
    A.dq = dq;
    A.dkey = dk_out;
    A.dval = dv_out;
    A.dg = dg;
    A.lddq = lddq;
    A.lddk = lddk;
    A.lddv = lddv;
    A.lddg = lddg;
    A.dh0 = dh0;
    LX_TRY(lx::attend_grad_launch(A, (int)type, gate_type == LAPLEX_F32 ? 0 : (int)type, (hipStream_t)stream),
           "attend backward");
    return LAPLEX_OK;
}

laplex_status laplex_attend_step(int64_t n, int64_t pool, const int32_t* slots, int64_t heads, int64_t query_heads,
                                 int64_t key_heads, int64_t value_heads, int64_t dk, int64_t dv, laplex_dtype type,
                                 laplex_dtype gate_type, float scale, const void* q, int64_t ldq, const void* k,
                                 int64_t ldk, const void* v, int64_t ldv, const void* g, int64_t ldg, float* state,
                                 void* y, int64_t ldy, void* stream)
{
    lx::AttendArgs sizes;  // a step's own limits: those of a pass of no rows
    if (!attend_sizes(sizes, 0, 1, heads, query_heads, key_heads, value_heads, dk, dv, type) || n < 0 ||
        n > 0x7FFFFFFF || pool < 0 || pool > 0x7FFFFFFF)
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, kBadAttend);
    if (gate_type != type && gate_type != LAPLEX_F32) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "bad gate_type");
    if (!slots && n > pool) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "without slots n must be at most pool");
    if (n * heads > (int64_t)1 << 37) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "n * heads must be at most 2^37");
    if (n == 0) return LAPLEX_OK;
    if (!q || !k || !v || !g || !y || (pool > 0 && !state))
        return fail(LAPLEX_ERR_INVALID_ARGUMENT, "q, k, v, g, state or y is NULL");
    const size_t e = dtype_size(type), eg = dtype_size(gate_type);
    const int64_t one = heads * dk * dv;
    const Rows outs[2] = {{y, n, ldy, heads * dv, e}, {state, pool, one, one, 4}};
    const Rows ins[5] = {{q, n, ldq, query_heads * dk, e}, {k, n, ldk, key_heads * dk, e},
                         {v, n, ldv, value_heads * dv, e}, {g, n, ldg, heads, eg}, {slots, 1, n, n, 4}};
    for (const Rows& r : {outs[0], outs[1], ins[0], ins[1], ins[2], ins[3], ins[4]})
        if (!rows_ok(r)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, "a bad row pitch or alignment");
    if (const char* m = check_outputs(outs, 2, ins, 5)) return fail(LAPLEX_ERR_INVALID_ARGUMENT, m);
    const laplex_status st = check_device();
    if (st != LAPLEX_OK) return st;
    lx::AttendStepArgs A;
    A.n = n;
    A.pool = pool;
    A.heads = (int)heads;
    A.hq = (int)query_heads;
    A.hk = (int)key_heads;
    A.hv = (int)value_heads;
    A.dk = (int)dk;
    A.dv = (int)dv;
    A.scale = scale;
    A.q = q;
    A.k = k;
    A.v = v;
    A.g = g;
    A.ldq = ldq;
    A.ldk = ldk;
    A.ldv = ldv;
    A.ldg = ldg;
    A.slots = slots;
    A.state = state;
    A.y = y;
    A.ldy = ldy;
    LX_TRY(lx::attend_step_launch(A, (int)type, gate_type == LAPLEX_F32 ? 0 : (int)type, (hipStream_t)stream),
           "attend step");
    return LAPLEX_OK;
}

}  // extern "C"
