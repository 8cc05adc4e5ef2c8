// The MoE operators and the token-scaled quantizer behind their own C-ABI on the
// CPU: the argument checks, the launch rules and every workgroup of every launch.
// A call runs in a child process.  Each buffer lies in pages of its own with a
// page that cannot be touched in front and behind, and ends (or begins) where
// that page does, so a plain load or store outside it ends the child, which
// says where.
#include <signal.h>
#include <sys/mman.h>
#include <sys/wait.h>
#include <unistd.h>

#include "moe_device.hpp"
#include "w8_block.hpp"
#include "w8_internal.hpp"
#include "w8_route.hpp"

namespace w8 {
// The library's own of w8_capi.cpp; no device is asked for.
std::string g_error;
w8_status fail(w8_status s, const std::string& msg) {
  g_error = msg;
  return s;
}
w8_status ok() { return W8_OK; }
std::string hip_msg(const char* what, hipError_t) { return what; }
w8_status check_device() { return W8_OK; }
uint8_t* g_dynamic_lds = nullptr;
}  // namespace w8

namespace {
constexpr size_t kPage = 4096, kText = 4096;
struct Buffer {
  std::string name;
  uint8_t *map, *p;
  size_t mapped, bytes;
};
std::vector<Buffer> g_buffers;
char* g_text = nullptr;
int g_lds_at_end = 1;

uint8_t* guarded(const char* name, size_t bytes, int at_end, int flags) {
  const size_t body = (bytes + kPage - 1) / kPage * kPage + (bytes ? 0 : kPage);
  uint8_t* map = (uint8_t*)mmap(nullptr, body + 2 * kPage, PROT_NONE, flags | MAP_ANONYMOUS, -1, 0);
  mprotect(map + kPage, body, PROT_READ | PROT_WRITE);
  uint8_t* p = map + kPage + (at_end ? body - bytes : 0);
  g_buffers.push_back({name, map, p, body + 2 * kPage, bytes});
  return p;
}
uint8_t* new_lds(size_t bytes) {
  // (it begins on 16 bytes)
  w8::g_dynamic_lds = guarded("dynamic LDS", (bytes + 15) / 16 * 16, g_lds_at_end, MAP_PRIVATE);
  return w8::g_dynamic_lds;
}
void on_fault(int, siginfo_t* info, void*) {
  const uint8_t* at = (const uint8_t*)info->si_addr;
  const Buffer* near = nullptr;
  for (const Buffer& b : g_buffers)
    if (at >= b.map && at < b.map + b.mapped) near = &b;
  const emu::Machine& g = emu::m();
  snprintf(g_text, kText, "access at %s + %lld (of %zu), block %u %u %u thread %d",
           near ? near->name.c_str() : "?", near ? (long long)(at - near->p) : (long long)(intptr_t)at,
           near ? near->bytes : 0, g.block, g.at.y, g.at.z, g.current);
  _exit(3);
}

template <class Args>
void one_block(const void* kernel, void** args) {
  reinterpret_cast<void (*)(Args)>(const_cast<void*>(kernel))(*static_cast<Args*>(args[0]));
}
void combine_block(const void* kernel, void** args) {
  reinterpret_cast<void (*)(w8::CombineArgs, int, int)>(const_cast<void*>(kernel))(
      *static_cast<w8::CombineArgs*>(args[0]), *static_cast<int*>(args[1]),
      *static_cast<int*>(args[2]));
}

// The call in a child: its status, or 100 + the number of faults.
int in_child(void (*thunk)(const void*, void**), int descending, const std::function<int()>& call) {
  if (!g_text)
    g_text = (char*)mmap(nullptr, kText, PROT_READ | PROT_WRITE, MAP_SHARED | MAP_ANONYMOUS, -1, 0);
  g_text[0] = 0;
  const pid_t child = fork();
  if (child == 0) {
    static char stack[65536];
    stack_t ss{};
    ss.ss_sp = stack;
    ss.ss_size = sizeof stack;
    sigaltstack(&ss, nullptr);
    struct sigaction sa {};
    sa.sa_sigaction = on_fault;
    sa.sa_flags = SA_SIGINFO | SA_ONSTACK;
    sigaction(SIGSEGV, &sa, nullptr);
    sigaction(SIGBUS, &sa, nullptr);
    emu::Machine& g = emu::m();
    g.opt.descending = descending;
    g.opt.partial = true;
    g.thunk = thunk;
    g.dynamic_lds = new_lds;
    g.ranges.clear();
    for (const Buffer& b : g_buffers) g.ranges.push_back({b.name.c_str(), b.p, b.bytes});
    const int status = call();
    if (status) snprintf(g_text, kText, "%s", w8::g_error.c_str());
    if (g.bad) snprintf(g_text, kText, "%s", g.text.c_str());
    _exit(g.bad ? 2 : status ? 10 + status : 0);
  }
  int how = 0;
  waitpid(child, &how, 0);
  return WIFEXITED(how) ? WEXITSTATUS(how) : 99;
}
}  // namespace

extern "C" {
void* emu_buffer(const char* name, long long bytes, int at_end) {
  return guarded(name, (size_t)bytes, at_end, MAP_SHARED);
}
void emu_free_all() {
  for (const Buffer& b : g_buffers) munmap(b.map, b.mapped);
  g_buffers.clear();
}
const char* emu_text() { return g_text; }
void emu_lds_at_end(int on) { g_lds_at_end = on; }

// 0, 10 + a refusal's status, 2: faults that the emulated device saw, 3: an
// access outside every buffer.
int emu_layer(int descending, int fmt, int E, int T, int topk, int D, int I, const void* xq,
              int64_t ldq, const float* sx, const int32_t* experts, const float* weights,
              const void* w1, int64_t ldw1, int64_t w1_stride, const float* s1, int64_t s1_stride,
              const void* w2, int64_t ldw2, int64_t w2_stride, const float* s2, int64_t s2_stride,
              const void* base, int64_t ldb, void* y, int64_t ldy, void* ws, int64_t ws_bytes) {
  return in_child(one_block<w8::MoeLayerArgs>, descending, [&] {
    return (int)w8_moe_layer((w8_fmt)fmt, E, T, topk, D, I, xq, ldq, sx, experts, weights, w1, ldw1,
                             w1_stride, s1, s1_stride, w2, ldw2, w2_stride, s2, s2_stride, base,
                             ldb, y, ldy, ws, (size_t)ws_bytes, nullptr);
  });
}
int emu_route(int descending, int T, int E, int topk, const void* logits, int64_t ldl, int fp32,
              int renormalize, float scale, int32_t* experts, float* weights, int32_t* offsets,
              int32_t* rows, int32_t* slots, void* ws, int64_t ws_bytes) {
  return in_child(one_block<w8::RouteArgs>, descending, [&] {
    return (int)w8_moe_route(T, E, topk, logits, ldl, fp32, renormalize, scale, experts, weights,
                             offsets, rows, slots, ws, (size_t)ws_bytes, nullptr);
  });
}
int emu_combine(int descending, int T, int topk, int D, const void* y, int64_t ldy, int n_rows,
                const float* weights, const int32_t* slots, const void* base, int64_t ldb,
                void* out, int64_t ldo) {
  return in_child(combine_block, descending, [&] {
    return (int)w8_moe_combine(T, topk, D, y, ldy, n_rows, weights, slots, base, ldb, out, ldo,
                               nullptr);
  });
}
int emu_quantize(int descending, int fmt, int M, int K, const void* x, int64_t ldx,
                 const void* gate, int64_t ldg, int reciprocal, void* xq, int64_t ldq, float* sx) {
  return in_child(one_block<w8::TokenQuantArgs>, descending, [&] {
    const w8::TokenQuantArgs a{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(gate),
                               static_cast<uint8_t*>(xq), sx, ldx, ldg, ldq, M, K, reciprocal};
    return (int)w8::launch_token_quantize(fmt, a, nullptr);
  });
}
long long emu_layer_workspace(int T, int topk, int D, int I) {
  size_t n = 0;
  return w8_moe_layer_workspace_size(T, topk, D, I, &n) ? -1 : (long long)n;
}
long long emu_route_workspace(int T, int E, int topk) {
  size_t n = 0;
  return w8_moe_route_workspace_size(T, E, topk, &n) ? -1 : (long long)n;
}
}
