// The kernel launches and the CUDA runtime calls that the library's entry points make, as fakes
// that write down what they are called with, so that a CPU test can drive the entry points: which
// kernels a call launches, on which stream, with how many splits and CTAs, and what it does when a
// launch fails.  Test infrastructure only: nothing in the library uses it.
#include <cstring>
#include <map>
#include <vector>

#include "pa_internal.h"

namespace {

struct Event {
    const char *name;
    int64_t stream, event;       // stream; event recorded or waited for
    int64_t value[4];            // splits, max_ctas and two more
};

std::vector<Event> g_events;
char g_fails[64] = "";
cudaError_t g_last = cudaSuccess;
int g_tensor_cores = 1;
std::map<int64_t, int64_t> g_capture, g_event_capture;      // of a stream, of the last record of an event (0: none)
int64_t g_handles = 0;

int64_t id(const void *p) { return (int64_t)reinterpret_cast<uintptr_t>(p); }

// Writes the call down, and fails where the test asked for it.
cudaError_t note(const char *name, cudaStream_t st, int64_t a = 0, int64_t b = 0, int64_t c = 0, int64_t d = 0, const void *event = nullptr) {
    const bool fails = !std::strcmp(name, g_fails);
    if (!fails) g_events.push_back({name, id(st), id(event), {a, b, c, d}});
    if (fails) g_last = cudaErrorInvalidValue;
    return fails ? cudaErrorInvalidValue : cudaSuccess;
}

}  // namespace

extern "C" {

void fake_reset(const char *fails, int tensor_cores) {
    g_events.clear();
    g_capture.clear();
    g_event_capture.clear();
    std::strncpy(g_fails, fails, sizeof g_fails - 1);
    g_tensor_cores = tensor_cores;
    g_last = cudaSuccess;
}
void fake_capture(int64_t stream, int64_t capture) { g_capture[stream] = capture; }
int fake_events() { return (int)g_events.size(); }
const char *fake_event(int i, int64_t *stream, int64_t *event, int64_t *value) {
    const Event &e = g_events[(size_t)i];
    *stream = e.stream;
    *event = e.event;
    std::memcpy(value, e.value, sizeof e.value);
    return e.name;
}

cudaError_t cudaGetDevice(int *dev) { return *dev = 0, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *value, cudaDeviceAttr, int) { return *value = 152, cudaSuccess; }
const char *cudaGetErrorString(cudaError_t) { return "a fake's error"; }
cudaError_t cudaGetLastError() {
    const cudaError_t e = g_last;
    return g_last = cudaSuccess, e;
}
cudaError_t cudaMemcpyAsync(void *, const void *, size_t, cudaMemcpyKind, cudaStream_t st) { return note("copy", st); }
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes *at, const void *) {
    std::memset(at, 0, sizeof *at);
    at->type = cudaMemoryTypeDevice;
    return cudaSuccess;
}
cudaError_t cudaStreamCreateWithFlags(cudaStream_t *st, unsigned) {
    return *st = reinterpret_cast<cudaStream_t>(0x1000 + ++g_handles), cudaSuccess;
}
cudaError_t cudaEventCreateWithFlags(cudaEvent_t *ev, unsigned) {
    return *ev = reinterpret_cast<cudaEvent_t>(0x1000 + ++g_handles), cudaSuccess;
}
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaStreamDestroy(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t st, cudaStreamCaptureStatus *s) {
    if (!std::strcmp("is_capturing", g_fails)) return g_last = cudaErrorStreamCaptureImplicit;
    return *s = g_capture[id(st)] ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone, cudaSuccess;
}
cudaError_t cudaStreamGetCaptureInfo(cudaStream_t st, cudaStreamCaptureStatus *s, unsigned long long *capture, cudaGraph_t *,
                                     const cudaGraphNode_t **, const cudaGraphEdgeData **, size_t *) {
    *capture = (unsigned long long)g_capture[id(st)];
    return cudaStreamIsCapturing(st, s);
}
cudaError_t cudaEventRecord(cudaEvent_t ev, cudaStream_t st) {
    g_event_capture[id(ev)] = g_capture[id(st)];
    return note("record", st, 0, 0, 0, 0, ev);
}
// A stream joins the capture of what it waits for; one that is in another capture may not.
cudaError_t cudaStreamWaitEvent(cudaStream_t st, cudaEvent_t ev, unsigned) {
    const int64_t capture = g_event_capture[id(ev)];
    if (g_capture[id(st)] && g_capture[id(st)] != capture) return cudaErrorStreamCaptureIsolation;
    g_capture[id(st)] = capture;
    return note("wait", st, 0, 0, 0, 0, ev);
}

}  // extern "C"

namespace pa {

cudaError_t read_device_status(int32_t *code, bool) { return *code = 0, cudaSuccess; }
int32_t *device_status_ptr() {
    static int32_t word;
    return &word;
}

bool prefill_supported(const AttnArgs &a) { return g_tensor_cores && a.d == 128 && a.dtype != PA_F32 && a.plan.n_tiles > 0; }
bool prefix_supported(const AttnArgs &a) { return g_tensor_cores && a.d == 128 && a.dtype != PA_F32; }
bool mla_supported(const AttnArgs &) { return g_tensor_cores != 0; }
bool q8_decode_tc_supported(const Q8AttnArgs &q) { return g_tensor_cores && q.a.dtype != PA_F32; }
bool mass_items_grouped(const MassArgs &, bool) { return true; }
bool evict_fits_grid(const EvictArgs &, bool) { return true; }

cudaError_t launch_kv_store(const PlanView &, const void *, const void *, void *, void *, int, int, int, int, cudaStream_t st) { return note("store", st); }
cudaError_t launch_decode(const AttnArgs &a, bool, cudaStream_t st) { return note("decode", st, a.splits, a.max_ctas, a.skip); }
cudaError_t launch_prefill(const AttnArgs &a, cudaStream_t st) { return note("prefill", st, a.splits, a.max_ctas, a.plan.pages); }
cudaError_t launch_prefix(const AttnArgs &a, int32_t shared, cudaStream_t st) { return note("prefix", st, a.splits, a.max_ctas, shared); }
cudaError_t launch_merge(const AttnArgs &a, bool use_list, cudaStream_t st) { return note("merge", st, a.splits, 0, use_list); }
cudaError_t launch_mla(const AttnArgs &a, bool, cudaStream_t st) { return note("mla", st, a.splits); }
cudaError_t launch_plan_advance(const PlanView &, int32_t *, cudaStream_t st) { return note("advance", st); }
cudaError_t launch_norm_rope_store(const NormRopeArgs &, cudaStream_t st) { return note("norm_rope_store", st); }
cudaError_t launch_mass_index(const MassArgs &, MassRecords, cudaStream_t st) { return note("mass_index", st); }
cudaError_t launch_lse_final(const MassArgs &, float *, cudaStream_t st) { return note("lse_final", st); }
cudaError_t launch_mass_items(const MassArgs &, bool, const AttnArgs *, bool, cudaStream_t st) { return note("mass_items", st); }
cudaError_t launch_mass_tiles_prepare(const MassArgs &, cudaStream_t st) { return note("mass_tiles_prepare", st); }
cudaError_t launch_mass_tiles(const MassArgs &, cudaStream_t st) { return note("mass_tiles", st); }
cudaError_t launch_mass_recompute(const MassArgs &, cudaStream_t st) { return note("mass_recompute", st); }
cudaError_t launch_evict(const EvictArgs &, int, int, bool, cudaStream_t st) { return note("evict", st); }
cudaError_t launch_q8_store(const Q8StoreArgs &, cudaStream_t st) { return note("q8_store", st); }
cudaError_t launch_q8_load(const Q8LoadArgs &, int longest, cudaStream_t st) { return note("q8_load", st, 0, 0, longest); }
cudaError_t launch_q8_places(const PlanView &, int2 *, int32_t window, int32_t, int32_t room, int32_t *, cudaStream_t st) {
    return note("q8_places", st, 0, 0, room, window);
}
cudaError_t launch_q8_decode_any(const Q8AttnArgs &q, bool, cudaStream_t st) { return note("q8_decode_any", st, q.a.splits, q.a.max_ctas); }
cudaError_t launch_q8_decode_tc(const Q8AttnArgs &q, bool, int, cudaStream_t st) { return note("q8_decode_tc", st, q.a.splits, q.a.max_ctas); }

}  // namespace pa
